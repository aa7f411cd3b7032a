// Gated delta rule, chunkwise forward. Per head, with a_t = exp(log decay):
//     S' = a_t S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,
//     o_t = scale S_t^T q_t.
// In blocks of 64 tokens, G_r the cumulative log decay of a block and
// E_rs = exp(G_r - G_s):
//     A_rs = beta_r E_rs (k_r . k_s)  (s < r),   T = (I + A)^-1,
//     V' = T X,   X = beta (V - e^G K S),
//     O = scale e^G Q S + P V',   P_rs = scale E_rs (q_r . k_s)  (s <= r),
//     S+ = e^(G_last) S + K^T (e^(G_last - G) V').
// Two launches: delta_prep_kernel forms T, P and the decay vectors of every
// block and head at once; delta_chain_kernel takes the state through a
// sequence's blocks, one workgroup per 32 or 64 value columns of a head, since
// the columns of S, V' and O do not meet.
#include "delta_common.hpp"

namespace ret {

constexpr float kMinBeta = 1e-20f;

constexpr int kPrepPitch = 68;

// 64 x 64 fp32 values in LDS to row-major planes of T (or their transpose);
// only the first `planes` planes are stored.
template <typename T, bool TRANS>
__device__ __forceinline__ void store_matrix(const float (*m)[kPrepPitch], T* out, int planes, int tid) {
  const int r = tid >> 2, c0 = (tid & 3) * 16;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + 8 * half + j;
      x[j] = TRANS ? m[c][r] : m[r][c];
    }
    for (int pl = 0; pl < planes; ++pl) {
      T* dst = out + pl * kB * kB + r * kB + c0 + 8 * half;
      F8 y;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y.x[j] = (float)(T)x[j];
        x[j] -= y.x[j];
      }
      store8(dst, y);
    }
  }
}

// One workgroup per (block, head). The products run on 16x16 tiles, wave w the
// rows 16 w .. + 15 and the columns up to them. T comes by blocks of 16: wave
// w inverts diagonal block w by forward substitution (lane = column), then
// takes block column w down: T_ij = -T_ii sum_k A_ik T_kj, in fp32 products.
// The cumulative decays are summed in 64 bits: E is the exponential of a
// difference of two sums that may both be large.
template <typename T, int D, bool GRAD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaParams p) {
  __shared__ double sg[kB];
  __shared__ float sbeta[kB];
  __shared__ __attribute__((aligned(16))) float sa[kB][kPrepPitch], st[kB][kPrepPitch], sp[kB][kPrepPitch];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6);
  const int b = blockIdx.x / p.blocks_max, blk = blockIdx.x % p.blocks_max, h = blockIdx.y;
  if (blockIdx.x == 0 && h == 0) {
    // control block: word 1 tells of packed bounds that had to be clamped
    bool ok = true;
    if (p.cu)
      for (int i = tid; i < p.batch; i += 256) {
        int t0, n;
        ok = clamp_span(p.cu[i], p.cu[i + 1], p.total, p.seqlen, t0, n) && ok;
      }
    ok = __syncthreads_and(ok);
    if (tid == 0) {
      p.ctrl[0] = 0;
      p.ctrl[1] = ok ? 0 : 2;
    }
  }
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  if (blk * kB >= len) return;
  const int rows = min(kB, len - blk * kB);
  const int64_t row0 = tok0 + blk * kB;
  const int64_t slot = (int64_t)(base + blk) * p.heads + h;

  if (w == 0) {
    float g = 0.f, be = 0.f;
    if (lane < rows) {
      g = p.log_decay[(row0 + lane) * p.heads + h];
      be = p.beta[(row0 + lane) * p.heads + h];
      if (g < kMinLogDecay) g = kMinLogDecay;
      // the backward divides by beta (d beta = dX . V' / beta): V' keeps its
      // relative accuracy under a tiny factor, and none under zero
      if (GRAD && fabsf(be) < kMinBeta) be = kMinBeta;
    }
    double s = g;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const double y = __shfl_up(s, o, 64);
      if (lane >= o) s += y;
    }
    sg[lane] = s;
    sbeta[lane] = be;
    const double last = __shfl(s, 63, 64);
    float* vec = p.vec + slot * (4 * kB);
    vec[lane] = (float)exp(s);
    vec[kB + lane] = (float)exp(last - s);
    vec[2 * kB + lane] = be;
  }

  const int g16 = lane >> 4, c = lane & 15;
  const int64_t qstride = (int64_t)p.k_heads * D;
  const int hk = h / (p.heads / p.k_heads);
  const T* Q = reinterpret_cast<const T*>(p.q) + row0 * qstride + hk * D + 8 * g16;
  const T* K = reinterpret_cast<const T*>(p.k) + row0 * qstride + hk * D + 8 * g16;
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) kk[ct] = qk[ct] = zero4();
  const int own = 16 * w + c;
#pragma unroll 2
  for (int ks = 0; ks < D / 32; ++ks) {
    const frag_t<T> fq = global_row8(Q + own * qstride + 32 * ks, own < rows);
    const frag_t<T> fk = global_row8(K + own * qstride + 32 * ks, own < rows);
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      if (ct > w) break;
      const int r = 16 * ct + c;
      const frag_t<T> fb = ct == w ? fk : global_row8(K + r * qstride + 32 * ks, r < rows);
      kk[ct] = mma(fk, fb, kk[ct]);
      qk[ct] = mma(fq, fb, qk[ct]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) {
    const int s = 16 * ct + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * w + 4 * g16 + i;
      const float e = s <= r ? __builtin_amdgcn_exp2f((float)((sg[r] - sg[s]) * 1.4426950408889634)) : 0.f;
      sa[r][s] = s < r ? sbeta[r] * e * kk[ct][i] : 0.f;
      sp[r][s] = s <= r ? p.scale * e * qk[ct][i] : 0.f;
      st[r][s] = 0.f;
    }
  }
  __syncthreads();
  {
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float y = r == c ? 1.f : 0.f;
#pragma unroll
      for (int s = 0; s < r; ++s) y -= sa[16 * w + r][16 * w + s] * x[s];
      x[r] = y;
    }
    if (g16 == 0) {
#pragma unroll
      for (int r = 0; r < 16; ++r) st[16 * w + r][16 * w + c] = x[r];
    }
  }
  __syncthreads();
  {
    // block column w; B operands are accumulators: contraction index 4 g + s
    f32x4 col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) col[0][i] = st[16 * w + 4 * g16 + i][16 * w + c];
#pragma unroll
    for (int n = 1; n < 4; ++n) {
      if (w + n > 3) break;
      const int ib = w + n;
      f32x4 m = zero4();
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(&sa[16 * ib + c][16 * (w + k) + 4 * g16]);
#pragma unroll
        for (int s = 0; s < 4; ++s) m = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], col[k][s], m, 0, 0, 0);
      }
      const f32x4 d = *reinterpret_cast<const f32x4*>(&st[16 * ib + c][16 * ib + 4 * g16]);
      f32x4 t = zero4();
#pragma unroll
      for (int s = 0; s < 4; ++s) t = __builtin_amdgcn_mfma_f32_16x16x4f32(-d[s], m[s], t, 0, 0, 0);
      col[n] = t;
#pragma unroll
      for (int i = 0; i < 4; ++i) st[16 * ib + 4 * g16 + i][16 * w + c] = t[i];
    }
  }
  __syncthreads();
  constexpr int NP = Planes<T>::N;
  store_matrix<T, false>(st, reinterpret_cast<T*>(p.t) + slot * (NP * kB * kB), NP, tid);
  // the forward's outputs are of type T: one plane of P (an error of 2^-9 of
  // the rounding that the output itself takes); the backward's row sums are
  // fp32 and take both
  constexpr int PP = GRAD ? NP : 1;
  store_matrix<T, false>(sp, reinterpret_cast<T*>(p.p) + slot * (PP * kB * kB), PP, tid);
  if constexpr (GRAD) {
    store_matrix<T, true>(st, reinterpret_cast<T*>(p.tt) + slot * (NP * kB * kB), NP, tid);
    store_matrix<T, true>(sp, reinterpret_cast<T*>(p.pt) + slot * (NP * kB * kB), NP, tid);
  }
}

// What a wave reads of a block before it can start on it.
template <typename T, int D, bool GRAD>
struct BlockIn {
  using CS = ChainShape<T, D>;
  static constexpr int NP = Planes<T>::N, PP = GRAD ? NP : 1;
  frag_t<T> k[2][4], q[2][4];       // rows of K and Q, the wave's 64 key columns
  frag_t<T> t[NP][2], p[PP][2];     // rows 16 w .. + 15 of T and P
  T v[CS::CG][4][2];                // the quarter's values
  T dout[GRAD ? CS::CG : 1][4][2];
  f32x4 eg, el, beta;
  float last;
};

template <typename T, int D, bool GRAD>
__device__ __forceinline__ void load_block(BlockIn<T, D, GRAD>& in, const DeltaParams& p, int64_t row0, int rows,
                                           int64_t slot, int h, int hk, int slice, int w, int lane) {
  using CS = ChainShape<T, D>;
  constexpr int NP = Planes<T>::N, PP = GRAD ? NP : 1;
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;
  const float* vec = p.vec + slot * (4 * kB);
  const T* tm = reinterpret_cast<const T*>(p.t) + slot * (NP * kB * kB) + (16 * w + c) * kB + 8 * g16;
  const T* pm = reinterpret_cast<const T*>(p.p) + slot * (PP * kB * kB) + (16 * w + c) * kB + 8 * g16;
  if (w < CS::WAVES) {
    const int64_t at = row0 * qs + hk * D + 64 * (w % CS::RG) + 8 * h2;
    const T* K = reinterpret_cast<const T*>(p.k) + at;
    const T* Q = reinterpret_cast<const T*>(p.q) + at;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int r = 32 * rt + n;
        in.k[rt][ks] = global_row8(K + r * qs + 16 * ks, r < rows);
        in.q[rt][ks] = global_row8(Q + r * qs + 16 * ks, r < rows);
      }
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (ks > (w >> 1)) break;  // T and P are lower triangular
#pragma unroll
    for (int pl = 0; pl < NP; ++pl) in.t[pl][ks] = global_row8(tm + pl * kB * kB + 32 * ks, true);
#pragma unroll
    for (int pl = 0; pl < PP; ++pl) in.p[pl][ks] = global_row8(pm + pl * kB * kB + 32 * ks, true);
  }
  const int r4 = 16 * w + 4 * g16;
  const T* V = reinterpret_cast<const T*>(p.v) + row0 * vs + h * D + slice * CS::SL + 2 * c;
  const T* DO = GRAD ? reinterpret_cast<const T*>(p.dout) + row0 * vs + h * D + slice * CS::SL + 2 * c : nullptr;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int cg = 0; cg < CS::CG; ++cg)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        in.v[cg][i][e] = r4 + i < rows ? V[(r4 + i) * vs + 32 * cg + e] : (T)0.f;
        if constexpr (GRAD) in.dout[cg][i][e] = r4 + i < rows ? DO[(r4 + i) * vs + 32 * cg + e] : (T)0.f;
      }
  in.eg = *reinterpret_cast<const f32x4*>(vec + r4);
  in.el = *reinterpret_cast<const f32x4*>(vec + kB + r4);
  in.beta = *reinterpret_cast<const f32x4*>(vec + 2 * kB + r4);
  in.last = vec[kB - 1];
}

// The state's way through one sequence's blocks, for SL value columns of one
// head; GRAD: the same walk for the backward, which keeps V', the states and
// the row sums o . dO in place of the output.
// A block takes three exchanges between the waves: each wave multiplies its 64
// key rows of S into K S (partial sums of all 64 tokens); a quarter of the
// tokens each, the waves add these up to X; V' = T X, a quarter each; then
// every wave adds K^T V' to its rows. Q S and P V' follow in the gaps.
template <typename T, int D, bool GRAD>
__global__ __launch_bounds__(256) void delta_chain_kernel(DeltaParams p) {
  using CS = ChainShape<T, D>;
  using KT = typename CS::KTile;
  constexpr int NP = Planes<T>::N, PP = GRAD ? NP : 1;
  T* const tag = nullptr;
  __shared__ __attribute__((aligned(1024))) char kt[CS::WAVES * KT::BYTES];
  __shared__ __attribute__((aligned(16))) f32x4 part_k[CS::WAVES * 512], part_q[CS::WAVES * 512];
  __shared__ __attribute__((aligned(16))) T ox[CS::OPND], ov[CS::OPND], ow[CS::OPND];

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6);
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int slice = id % CS::NSL, bh = id / CS::NSL, h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.k_heads);
  const int rg = w % CS::RG, cg_w = w / CS::RG;
  const bool holds = w < CS::WAVES;
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  const int nblk = (len + kB - 1) / kB;
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;

  // the state's element (tile t, i): key row krow + 32 t + state_row(i, h2),
  // value column vcol
  const int krow = 64 * rg, vcol = slice * CS::SL + 32 * cg_w + n;
  f32x16 s[2] = {zero16(), zero16()};
  if (holds && p.state_in) {
    const float* si = p.state_in + (int64_t)bh * D * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = si[(krow + 32 * t + state_row(i, h2)) * D + vcol];
  }

  char* my_kt = kt + w * KT::BYTES;
  TileLoads<T, KT, 1> loads;
  loads.init(qs, lane);
  // bf16 reads a block ahead; the fp32 operands do not fit the registers twice
  constexpr bool kAhead = sizeof(T) == 2;
  BlockIn<T, D, GRAD> in;
  if (kAhead && nblk)
    load_block<T, D, GRAD>(in, p, tok0, min(kB, len), (int64_t)base * p.heads + h, h, hk, slice, w, lane);

  for (int blk = 0; blk < nblk; ++blk) {
    const int64_t row0 = tok0 + (int64_t)blk * kB;
    const int rows = min(kB, len - blk * kB);
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    if constexpr (!kAhead) load_block<T, D, GRAD>(in, p, row0, rows, slot, h, hk, slice, w, lane);
    f32x16 qsum[2] = {zero16(), zero16()};
    if (holds) {
      // K's tile for the state's update, read after the third exchange
      const T* Kt = reinterpret_cast<const T*>(p.k) + row0 * qs + hk * D + krow;
      __builtin_amdgcn_s_waitcnt(kWaitLds);  // the last block's reads of the tile
      if (rows == kB)
        loads.issue(my_kt, Kt, qs, 0, 0);
      else
        loads.issue_clamped(my_kt, Kt, qs, 0, rows - 1, 0);
      f32x16 ksum[2] = {zero16(), zero16()};
#pragma unroll
      for (int t = 0; t < 2; ++t)
        static_for<2>([&](auto sl) {
          constexpr int SLI = decltype(sl)::value;
          const Split<T> f = split_acc<SLI>(s[t], tag);
          const int ks = 2 * t + SLI;
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) ksum[rt] = mma32(in.k[rt][ks], f.f[pl], ksum[rt]);
#pragma unroll
            for (int pl = 0; pl < PP; ++pl) qsum[rt] = mma32(in.q[rt][ks], f.f[pl], qsum[rt]);
          }
          if constexpr (GRAD) {
            // the state at the block's start, [dv][dk], for the gradients of q and k
            T* sn = reinterpret_cast<T*>(p.snap) + (slot * D + vcol) * D + krow + 32 * t + 16 * SLI + 8 * h2;
            *reinterpret_cast<frag_t<T>*>(sn) = f.f[0];
          }
        });
      if constexpr (GRAD) {
        if (blk && blk % kDeltaGroup == 0) {
          float* an = p.anchor + ((((int64_t)(base / kDeltaGroup + b + blk / kDeltaGroup - 1) * p.heads + h) * CS::NSL +
                                   slice) * CS::WAVES + w) * 2048 + lane * 4;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<f32x4*>(an + (4 * t + q) * 256) =
                  f32x4{s[t][4 * q], s[t][4 * q + 1], s[t][4 * q + 2], s[t][4 * q + 3]};
        }
      }
      put_partial(part_k, w, ksum, lane);
    }
    __syncthreads();

    // X of rows 16 w + 4 g16 + i
#pragma unroll
    for (int ct = 0; ct < CS::CT; ++ct) {
      const f32x4 ks = get_partial<CS::RG>(part_k, ct, 4 * w + g16, c);
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = in.beta[i] * ((float)in.v[ct >> 1][i][ct & 1] - in.eg[i] * ks[i]);
        x[i] = 16 * w + 4 * g16 + i < rows ? y : 0.f;
      }
      put_opnd<CS::PITCH, CS::OPLANE>(ox, 16 * ct + c, 16 * w + 4 * g16, x);
    }
    if (holds) put_partial(part_q, w, qsum, lane);
    __syncthreads();

    // V' = T X
    f32x4 u[CS::CT];
#pragma unroll
    for (int ct = 0; ct < CS::CT; ++ct) {
      u[ct] = zero4();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > (w >> 1)) break;
        frag_t<T> tf[NP], xf[NP];
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
          tf[pl] = in.t[pl][ks];
          xf[pl] = lds_row8(ox + pl * CS::OPLANE + (16 * ct + c) * CS::PITCH + 32 * ks + 8 * g16);
        }
        u[ct] = mma_split2(tf, xf, u[ct], tag);
      }
      put_opnd<CS::PITCH, CS::OPLANE>(ov, 16 * ct + c, 16 * w + 4 * g16, u[ct]);
      f32x4 ud;
#pragma unroll
      for (int i = 0; i < 4; ++i) ud[i] = u[ct][i] * in.el[i];
      put_opnd<CS::PITCH, CS::OPLANE>(ow, 16 * ct + c, 16 * w + quad_place(g16), ud);
    }
    const float last = in.last;
    __builtin_amdgcn_s_waitcnt(0);  // the K tile (LDS loads run past the compiler's counting)
    __syncthreads();

    // the next block's reads overlap the state's update
    BlockIn<T, D, GRAD> nx;
    if (kAhead && blk + 1 < nblk)
      load_block<T, D, GRAD>(nx, p, row0 + kB, min(kB, len - (blk + 1) * kB), slot + p.heads, h, hk, slice, w, lane);

    if (holds) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] *= last;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        frag_t<T> uf[NP];
#pragma unroll
        for (int pl = 0; pl < NP; ++pl)
          uf[pl] = lds_row8(ow + pl * CS::OPLANE + (32 * cg_w + col_place(n)) * CS::PITCH + 16 * ks + 8 * h2);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const frag_t<T> kf = state_col8<KT>(my_kt, 16 * ks, 32 * t, lane, tag);
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) s[t] = mma32(kf, uf[pl], s[t]);
        }
      }
    }
    // O of the quarter
    f32x4 dot = zero4();
#pragma unroll
    for (int cg = 0; cg < CS::CG; ++cg) {
      f32x4 o2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ct = 2 * cg + e;
        f32x4 o = get_partial<CS::RG>(part_q, ct, 4 * w + g16, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= p.scale * in.eg[i];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (ks > (w >> 1)) break;
          frag_t<T> vf[NP];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
            vf[pl] = lds_row8(ov + pl * CS::OPLANE + (16 * ct + c) * CS::PITCH + 32 * ks + 8 * g16);
          if constexpr (GRAD) {
            frag_t<T> pf[NP];
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) pf[pl] = in.p[pl][ks];
            o = mma_split2(pf, vf, o, tag);
          } else {
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) o = mma(in.p[0][ks], vf[pl], o);
          }
        }
        o2[e] = o;
        if constexpr (GRAD) {
#pragma unroll
          for (int i = 0; i < 4; ++i) dot[i] += o[i] * (float)in.dout[cg][i][e];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * w + 4 * g16 + i;
        if (r >= rows) continue;
        const int64_t at = (row0 + r) * vs + h * D + slice * CS::SL + 32 * cg + 2 * c;
        if constexpr (!GRAD) {
          T* o = reinterpret_cast<T*>(p.o) + at;
          o[0] = (T)o2[0][i];
          o[1] = (T)o2[1][i];
        } else {
          // V' in planes of whole tensors
          const int64_t plane = (int64_t)p.total * vs;
          T* uo = reinterpret_cast<T*>(p.u) + at;
          float r0 = u[2 * cg][i], r1 = u[2 * cg + 1][i];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) {
            const T a0 = (T)r0, a1 = (T)r1;
            uo[pl * plane] = a0;
            uo[pl * plane + 1] = a1;
            r0 -= (float)a0;
            r1 -= (float)a1;
          }
        }
      }
    }
    if constexpr (GRAD) {
#pragma unroll
      for (int i = 0; i < 4; ++i) dot[i] = sum16(dot[i]);
      if (c == 0) *reinterpret_cast<f32x4*>(p.odo + (slot * CS::NSL + slice) * kB + 16 * w + 4 * g16) = dot;
    }
    if (kAhead && blk + 1 < nblk) in = nx;
  }

  if (holds && p.state_out) {
    float* so = p.state_out + (int64_t)bh * D * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) so[(krow + 32 * t + state_row(i, h2)) * D + vcol] = s[t][i];
  }
  if constexpr (GRAD) {
    if (holds && nblk && p.d_state_out) {  // the last group's copy: only a gradient of the final state meets it
      float* an = p.anchor + ((((int64_t)(base / kDeltaGroup + b + (nblk - 1) / kDeltaGroup) * p.heads + h) * CS::NSL +
                               slice) * CS::WAVES + w) * 2048 + lane * 4;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4*>(an + (4 * t + q) * 256) =
              f32x4{s[t][4 * q], s[t][4 * q + 1], s[t][4 * q + 2], s[t][4 * q + 3]};
    }
  }
}

template <typename T, int D, bool GRAD>
static hipError_t launch_forward(const DeltaParams& p, hipStream_t stream) {
  using CS = ChainShape<T, D>;
  hipLaunchKernelGGL((delta_prep_kernel<T, D, GRAD>), dim3(p.batch * p.blocks_max, p.heads), dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_chain_kernel<T, D, GRAD>), dim3(CS::NSL * p.batch * p.heads), dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <typename T, int D>
static hipError_t launch_either(const DeltaParams& p, bool grad, hipStream_t stream) {
  return grad ? launch_forward<T, D, true>(p, stream) : launch_forward<T, D, false>(p, stream);
}

hipError_t launch_delta_forward(const DeltaParams& p, int d, int dtype, bool grad, hipStream_t stream) {
  if (dtype == 1) {
    switch (d) {
      case 64: return launch_either<bf16, 64>(p, grad, stream);
      case 128: return launch_either<bf16, 128>(p, grad, stream);
      case 256: return launch_either<bf16, 256>(p, grad, stream);
    }
  } else {
    switch (d) {
      case 64: return launch_either<float, 64>(p, grad, stream);
      case 128: return launch_either<float, 128>(p, grad, stream);
      case 256: return launch_either<float, 256>(p, grad, stream);
    }
  }
  return hipErrorInvalidValue;
}

hipError_t launch_delta_fwd(const DeltaParams& p, int d, int dtype, hipStream_t stream) {
  return launch_delta_forward(p, d, dtype, false, stream);
}

template <typename T, int D>
static void chain_layout(DeltaLayout& l) {
  l.slices = ChainShape<T, D>::NSL;
  l.planes = Planes<T>::N;
  l.mat_plane = kB * kB * sizeof(T);
}

DeltaLayout delta_layout(int batch, int seqlen, int d, int dtype, bool packed, int total) {
  DeltaLayout l;
  const size_t per = ((size_t)seqlen + kB - 1) / kB;
  l.blocks = packed ? (size_t)total / kB + batch : per * batch;
  // group g of a sequence is numbered (its first block) / kDeltaGroup + its place in the batch + g
  l.groups = l.blocks / kDeltaGroup + batch + 1;
  if (dtype == 1) {
    if (d == 64) chain_layout<bf16, 64>(l);
    else if (d == 128) chain_layout<bf16, 128>(l);
    else chain_layout<bf16, 256>(l);
  } else {
    if (d == 64) chain_layout<float, 64>(l);
    else if (d == 128) chain_layout<float, 128>(l);
    else chain_layout<float, 256>(l);
  }
  return l;
}

}  // namespace ret
