// Gated delta rule, chunkwise forward. Per head, with a_t = exp(log decay):
//     S' = a_t S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,
//     o_t = scale S_t^T q_t.
// In blocks of 64 tokens, G_r the cumulative log decay of a block and
// E_rs = exp(G_r - G_s):
//     A_rs = beta_r E_rs (k_r . k_s)  (s < r),   T = (I + A)^-1 diag(beta),
//     V' = T X,   X = V - e^G K S,
//     O = scale e^G Q S + P V' = scale e^G Q S + M X,   M = P T,
//     P_rs = scale E_rs (q_r . k_s)  (s <= r),
//     S+ = e^(G_last) S + K^T (e^(G_last - G) V').
// Two launches: delta_prep_kernel forms T, M and the decay vectors of every
// block and head at once; delta_chain_kernel takes the state through a
// sequence's blocks, one workgroup per 32 or 64 value columns of a head, since
// the columns of S, V' and O do not meet.
#include "delta_common.hpp"

namespace ret {

constexpr float kMinBeta = 1e-12f;

constexpr int kPrepPitch = 68;

// A 64 x 64 matrix in LDS (or its transpose) as row fragments of T in planes;
// only the first `planes` planes are stored.
template <typename T, bool TRANS>
__device__ __forceinline__ void store_matrix(const float (*m)[kPrepPitch], T* out, int planes, int tid) {
  const int lane = tid & 63;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = (tid >> 6) + 4 * i;
    const int r = 16 * (f >> 1) + (lane & 15), c = 32 * (f & 1) + 8 * (lane >> 4);
    F8 x, y;
    if constexpr (TRANS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x.x[j] = m[c + j][r];
    } else {
      x = load8(&m[r][c]);
    }
    for (int pl = 0; pl < planes; ++pl) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y.x[j] = (float)(T)x.x[j];
        x.x[j] -= y.x[j];
      }
      store8(out + mat_frag(pl, f >> 1, f & 1) + 8 * lane, y);
    }
  }
}

// One workgroup per (block, key head). K K^T and Q K^T run on 16x16 tiles, wave
// w the rows 16 w .. + 15 and the columns up to them, from rows staged in LDS
// by 128 columns, which also leave in the lanes' order. Then, for each value
// head, T by blocks of 16: wave w inverts diagonal block w by forward
// substitution (lane = column), then takes block column w down: T_ij = -T_ii
// sum_k A_ik T_kj, in fp32 products; the columns take their beta at the end.
// The cumulative decays are summed in 64 bits: E is the exponential of a
// difference of two sums that may both be large.
// All blocks at once, so bound by what passes: 158 us for 4096 blocks of bf16
// keys of 256 (268 MB read, 540 MB written: 5.1 TB/s, where a large copy
// reaches 5.2); 99 us for 32 value heads of 128 over 10287 packed tokens. A
// short sequence sees one block's latency, 13 us.
template <typename T, int D, bool GRAD>
__global__ __launch_bounds__(256, sizeof(T) == 4 && D > 64 ? 2 : 3) void delta_prep_kernel(DeltaParams p) {
  constexpr int HALF = D < 128 ? D : 128;  // columns staged at a time
  constexpr int SP = HALF + 16 / (int)sizeof(T);
  struct Stage { T k[kB][SP], q[kB][SP]; };
  struct Mats { float a[kB][kPrepPitch], t[kB][kPrepPitch], p[kB][kPrepPitch]; };
  union Shared { Stage st; Mats m; __device__ Shared() {} };
  __shared__ __attribute__((aligned(16))) Shared sh;
  __shared__ double sg[kB];
  __shared__ __attribute__((aligned(16))) float sbeta[kB];
  const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6);
  const int b = blockIdx.x / p.blocks_max, blk = blockIdx.x % p.blocks_max, hk = blockIdx.y;
  if (blockIdx.x == 0 && hk == 0) {
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
  const int g16 = lane >> 4, c = lane & 15;

  f32x4 kk[4], qk[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) kk[ct] = qk[ct] = zero4();
  {
    const int64_t stride = (int64_t)p.k_heads * D;
    const T* Q = reinterpret_cast<const T*>(p.q) + row0 * stride + hk * D;
    const T* K = reinterpret_cast<const T*>(p.k) + row0 * stride + hk * D;
    const int64_t out = ((int64_t)(base + blk) * p.k_heads + hk) * (kB * D) + 8 * lane;
    T* KF = reinterpret_cast<T*>(p.kf) + out;
    T* KC = reinterpret_cast<T*>(p.kc) + out;
    T* QF = reinterpret_cast<T*>(p.qf) + out;
    T* QC = reinterpret_cast<T*>(p.qc) + out;
    constexpr int CPR = HALF / 8;  // chunks of 8 elements in a staged row
    Raw8<T> rk[kB * CPR / 256], rq[kB * CPR / 256];
    auto load = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kB * CPR / 256; ++i) {
        const int r = (tid + 256 * i) / CPR, at = (tid + 256 * i) % CPR * 8;
        if (r < rows) {
          rk[i] = ld_raw8(K + r * stride + c0 + at);
          rq[i] = ld_raw8(Q + r * stride + c0 + at);
        } else {
          rk[i] = rq[i] = Raw8<T>{};
        }
      }
    };
    load(0);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += HALF) {
      if (c0) __syncthreads();
#pragma unroll
      for (int i = 0; i < kB * CPR / 256; ++i) {
        const int r = (tid + 256 * i) / CPR, at = (tid + 256 * i) % CPR * 8;
        st_raw8(&sh.st.k[r][at], rk[i], true);
        st_raw8(&sh.st.q[r][at], rq[i], true);
      }
      __syncthreads();
      if (c0 + HALF < D) load(c0 + HALF);
      // (a loop for each wave's number of tiles: no branch stands between products)
      auto products = [&](auto tiles) {
#pragma unroll 2
        for (int ks = 0; ks < HALF / 32; ++ks) {
          const frag_t<T> fq = lds_row8(&sh.st.q[16 * w + c][32 * ks + 8 * g16]);
          const frag_t<T> fk = lds_row8(&sh.st.k[16 * w + c][32 * ks + 8 * g16]);
          if constexpr (!GRAD) *reinterpret_cast<frag_t<T>*>(QF + query_frag<D>(w, c0 / 32 + ks)) = fq;
#pragma unroll
          for (int ct = 0; ct < decltype(tiles)::value; ++ct) {
            const frag_t<T> fb = lds_row8(&sh.st.k[16 * ct + c][32 * ks + 8 * g16]);
            kk[ct] = mma(fk, fb, kk[ct]);
            qk[ct] = mma(fq, fb, qk[ct]);
          }
        }
      };
      if (w == 0) products(std::integral_constant<int, 1>{});
      else if (w == 1) products(std::integral_constant<int, 2>{});
      else if (w == 2) products(std::integral_constant<int, 3>{});
      else products(std::integral_constant<int, 4>{});
#pragma unroll
      for (int i = 0; i < HALF / 32; ++i) {
        const int f = w + 4 * i;
        *reinterpret_cast<frag_t<T>*>(KF + key_frag(c0 / 16 + f / 2, f & 1)) =
            lds_row8(&sh.st.k[32 * (f & 1) + (lane & 31)][16 * (f / 2) + 8 * (lane >> 5)]);
      }
#pragma unroll
      for (int t = 0; t < HALF / 32; ++t) {
        *reinterpret_cast<frag_t<T>*>(KC + column_frag(c0 / 32 + t, w)) =
            state_col8(&sh.st.k[0][0], SP, 16 * w, 32 * t, lane);
        if constexpr (GRAD)
          *reinterpret_cast<frag_t<T>*>(QC + column_frag(c0 / 32 + t, w)) =
              state_col8(&sh.st.q[0][0], SP, 16 * w, 32 * t, lane);
      }
    }
  }

  if constexpr (GRAD) {
    float* pairs = p.pairs + ((int64_t)(base + blk) * p.k_heads + hk) * (2 * kB * kB);
#pragma unroll
    for (int ct = 0; ct < 4; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (16 * w + 4 * g16 + i) * kB + 16 * ct + c;
        pairs[at] = qk[ct][i];
        pairs[kB * kB + at] = kk[ct][i];
      }
  }

  const int group = p.heads / p.k_heads;
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    float (*const sa)[kPrepPitch] = sh.m.a;
    float (*const st)[kPrepPitch] = sh.m.t;
    float (*const sp)[kPrepPitch] = sh.m.p;
    __syncthreads();  // the staged rows, or the last head's matrices, have been read
    if (w == 0) {
      float g = 0.f, be = 0.f;
      if (lane < rows) {
        g = p.log_decay[(row0 + lane) * p.heads + h];
        be = p.beta[(row0 + lane) * p.heads + h];
        if (g < kMinLogDecay) g = kMinLogDecay;
        // the backward divides by beta (d beta = dv . V' / beta^2): dv and V'
        // keep their relative accuracy under a tiny factor, and none under zero
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
    for (int i = tid; i < kB * kB / 4; i += 256) {
      f32x4* at = reinterpret_cast<f32x4*>(&st[i / 16][i % 16 * 4]);
      *at *= *reinterpret_cast<const f32x4*>(&sbeta[i % 16 * 4]);
    }
    __syncthreads();
    if constexpr (!GRAD) {
      // M = P T, five products of 16x16 blocks a wave
      auto block = [&](int ib, int jb) {
        f32x4 m = zero4();
        for (int k = jb; k <= ib; ++k) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(&sp[16 * ib + c][16 * k + 4 * g16]);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            m = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], st[16 * k + 4 * g16 + s][16 * jb + c], m, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[16 * ib + 4 * g16 + i][16 * jb + c] = m[i];
      };
      if (w == 0) {
        block(3, 0);
        block(0, 0);
      } else if (w == 1) {
        block(3, 1);
        block(1, 0);
      } else if (w == 2) {
        block(2, 0);
        block(3, 2);
      } else {
        block(2, 1);
        block(1, 1);
        block(2, 2);
        block(3, 3);
      }
    }
    constexpr int NM = MatPlanes<T, GRAD>::N;
    store_matrix<T, false>(st, reinterpret_cast<T*>(p.t) + slot * (NM * kB * kB), NM, tid);
    if constexpr (GRAD) {
      store_matrix<T, true>(st, reinterpret_cast<T*>(p.tt) + slot * (NM * kB * kB), NM, tid);
      store_matrix<T, true>(sp, reinterpret_cast<T*>(p.pt) + slot * (NM * kB * kB), NM, tid);
    } else {
      __syncthreads();
      // all planes of M, as of T: with one, its rounding (2^-9) and that of a state
      // copied in one plane put o 2.4e-3 off where its own rounding gives 1.7e-3;
      // with two o is at its rounding, for 6% of the call (519 -> 552 us for 2 x 8192
      // tokens, 16 heads of 256)
      store_matrix<T, false>(sa, reinterpret_cast<T*>(p.m) + slot * (NM * kB * kB), NM, tid);
    }
  }
}

// The state's way through one sequence's blocks, for SL value columns of one
// head; GRAD: the same walk for the backward, which keeps V' and the states in
// place of the output.
// Bound by the way from one block's state to the next, which takes three
// exchanges between the four state waves: each multiplies its key rows of S
// into K S (partial sums of all 64 tokens); a quarter of the tokens each, they
// add these up to X; V' = T X, a quarter each; then every wave adds K^T V' to
// its rows. The other four waves follow with the output, a quarter of the
// tokens each: Q S from a copy of the state in LDS, and M X.
// The caches' 64 bytes a clock and LDS (writes at half the rate of reads) are
// nearly as busy as the matrix cores. So keys come as fragments from memory
// both ways round, not through a tile in LDS, and what a block reads is asked
// for a block ahead, spread over the step: a wave that asks for much at once
// waits until the caches have taken it.
// Measured: 423 us for 128 blocks a sequence of 256 x 256 states, 3.3 us a
// block; 256 workgroups of 32 columns, one a CU. 355 us for 65 blocks at most
// of 128 x 128 states (two workgroups a CU, 128 registers a lane). A block's 6.8
// MFLOP of a workgroup are 0.7 us at a CU's dense rate and its 124 KB 0.8 us at
// the caches' 64 bytes a clock: the rest is latency at the exchanges. X and V'
// by all eight waves: slower (T read twice); keys as a tile in LDS: slower (LDS
// writes); asking two blocks ahead: 491 us.
template <typename T, int D, bool GRAD>
__global__ __launch_bounds__(512, D == 128 && !GRAD ? 4 : 2) void delta_chain_kernel(DeltaParams p) {
  using CS = ChainShape<T, D>;
  constexpr int NP = Planes<T>::N, SZ = sizeof(T);
  constexpr int NM = MatPlanes<T, GRAD>::N;
  constexpr int RG = CS::RG, TPW = CS::TPW, CT = CS::CT, CG = CS::CG, PITCH = CS::PITCH, OPLANE = CS::OPLANE;
  // Two copies of the state let Q S wait until the state waves are back at
  // their products. fp32 has no room for the second, nor have two workgroups of
  // 128 columns a CU: they take Q S between the first two exchanges.
  constexpr bool kTwoCopies = SZ == 2 && !(D == 128 && !GRAD);
  constexpr bool kAhead = SZ == 2;  // fp32 keys do not fit the registers a block ahead
  constexpr int COPY = CS::SPLANE * NP;
  T* const tag = nullptr;
  __shared__ __attribute__((aligned(16))) f32x4 part[4 * 512];
  __shared__ __attribute__((aligned(16))) T ox[OPLANE * NM], ow[CS::OPND], ov[GRAD ? CS::OPND : 16];
  __shared__ __attribute__((aligned(16))) T os[COPY * (kTwoCopies ? 2 : 1)];

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_i(tid >> 6), w = wave & 3;
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int slice = id % CS::NSL, bh = id / CS::NSL, h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.k_heads);
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  const int r4 = 16 * w + 4 * g16;  // the lane's four tokens of the wave's quarter
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  const int nblk = (len + kB - 1) / kB;
  const int64_t vs = (int64_t)p.heads * D;
  const uint32_t vrow = (uint32_t)vs * SZ;
  // descriptors of block blk (no rows: nothing is read)
  auto rows_of = [&](int blk) { return blk < nblk ? min(kB, len - blk * kB) : 0; };
  auto key_rsrc = [&](const void* x, int blk) {  // keys or queries in the lanes' order
    return scalar_rsrc(reinterpret_cast<const T*>(x) + ((int64_t)(base + blk) * p.k_heads + hk) * (kB * D),
                       blk < nblk ? kB * D * SZ : 0);
  };
  auto value_rsrc = [&](const void* x, int blk) {
    return scalar_rsrc(reinterpret_cast<const T*>(x) + (tok0 + (int64_t)blk * kB) * vs + h * D, rows_of(blk) * vrow);
  };
  auto slot_of = [&](int blk) { return (int64_t)(base + blk) * p.heads + h; };
  auto mat_rsrc = [&](const void* x, int planes, int blk) {
    return scalar_rsrc(reinterpret_cast<const T*>(x) + slot_of(blk) * (planes * kB * kB),
                       blk < nblk ? planes * kB * kB * SZ : 0);
  };
  auto vec_rsrc = [&](int blk) { return scalar_rsrc(p.vec + slot_of(blk) * (4 * kB), blk < nblk ? 4 * kB * 4 : 0); };
  const uint32_t lane_off = 8 * lane * SZ;
  uint32_t pair_off[4];  // the lane's pairs of value columns, token i
#pragma unroll
  for (int i = 0; i < 4; ++i) pair_off[i] = (r4 + i) * vrow + (slice * CS::SL + 2 * c) * SZ;

  if (wave < 4) {
    const int rg = w % RG, cg = w / RG;
    // the state's element (tile t, i): key row krow + 32 t + state_row(i, h2), value column vcol
    const int krow = CS::KR * rg, vcol = slice * CS::SL + 32 * cg + n;
    f32x16 s[TPW];
#pragma unroll
    for (int t = 0; t < TPW; ++t) s[t] = zero16();
    // A first token that forgets starts from zeros whatever the state holds (a factor
    // of zero would keep a NaN or an infinity); an empty sequence passes it on.
    if (p.state_in && (nblk == 0 || p.vec[slot_of(0) * (4 * kB)] != 0.f)) {
      const float* si = p.state_in + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = si[(krow + 32 * t + state_row(i, h2)) * D + vcol];
    }
    T* my_os = os + (32 * cg + col_place(n)) * CS::SPITCH + krow + 8 * h2;

    frag_t<T> kf[2][CS::KS], kc[TPW][4], tf[2][NM];
#pragma unroll
    for (int pl = 0; pl < NM; ++pl) tf[1][pl] = zero_frag<T>();
    PairOf<T> v[CG][4];
    f32x4 eg, el;
    float last;
    auto load_keys = [&](int blk, int rt) {
      const auto rs = key_rsrc(p.kf, blk);
#pragma unroll
      for (int ks = 0; ks < CS::KS; ++ks)
        kf[rt][ks] = buf_frag(rs, lane_off, key_frag(CS::KS * rg + ks, rt) * SZ, tag);
    };
    auto load_column = [&](__amdgpu_buffer_rsrc_t rs, int t, int ks) {
      kc[t][ks] = buf_frag(rs, lane_off, column_frag(TPW * rg + t, ks) * SZ, tag);
    };
    auto load_values = [&](int blk) {  // what X takes
      const auto vr = value_rsrc(p.v, blk);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < CG; ++g) v[g][i] = buf_pair(vr, pair_off[i] + 32 * g * SZ, tag);
      eg = buf_f4(vec_rsrc(blk), r4 * 4, 0);
    };
    auto load_rest = [&](int blk) {  // what V' takes
      const auto tr = mat_rsrc(p.t, NM, blk);
#pragma unroll
      for (int pl = 0; pl < NM; ++pl)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= (w >> 1)) tf[ks][pl] = buf_frag(tr, lane_off, mat_frag(pl, w, ks) * SZ, tag);  // lower triangular
      const auto er = vec_rsrc(blk);
      el = buf_f4(er, r4 * 4, kB * 4);
      last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(er, 0, (kB - 1) * 4, 0));
    };
    load_values(0);
    load_rest(0);
    if constexpr (kAhead) {
      load_keys(0, 0);
      load_keys(0, 1);
    }

    for (int blk = 0; blk < nblk; ++blk) {
      if constexpr (!kAhead) {
        load_keys(blk, 0);
        load_keys(blk, 1);
      }
      const auto columns = key_rsrc(p.kc, blk);
      T* copy = my_os + (kTwoCopies ? (blk & 1) * COPY : 0);
      // K S: the first 32 tokens' products follow the state's rounding, their
      // sums go to LDS under the other 32 tokens' products
      Split<T> f[CS::KS];
      f32x16 ksum[2] = {zero16(), zero16()};
#pragma unroll
      for (int t = 0; t < TPW; ++t)
        static_for<2>([&](auto sl) {
          constexpr int SLI = decltype(sl)::value;
          const int ks = 2 * t + SLI;
          f[ks] = split_acc<SLI>(s[t], tag);
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) ksum[0] = mma32(kf[0][ks], f[ks].f[pl], ksum[0]);
          if constexpr (kAhead) {
            load_column(columns, t, 2 * SLI);
            load_column(columns, t, 2 * SLI + 1);
          }
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
            *reinterpret_cast<frag_t<T>*>(copy + pl * CS::SPLANE + 16 * ks) = f[ks].f[pl];
        });
      if constexpr (TPW > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int ks = 0; ks < CS::KS; ++ks)
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) ksum[1] = mma32(kf[1][ks], f[ks].f[pl], ksum[1]);
      put_partial(part, w, 0, ksum[0], lane);
      if constexpr (TPW > 1) __builtin_amdgcn_sched_barrier(0);
      put_partial(part, w, 1, ksum[1], lane);
      lds_barrier();

      // X of the quarter (zero behind the sequence's end: K and V are)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 x = -eg * get_partial<RG>(part, ct, 4 * w + g16, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += v[ct >> 1][i].get(ct & 1);
        put_opnd<PITCH, OPLANE, NM>(ox, row_of(ct, c), r4, x);
      }
      if constexpr (kAhead) load_keys(blk + 1, 0);
      load_values(blk + 1);
      lds_barrier();

      // V' of the quarter (waves 0 and 1 multiply T's upper zeros too, rather than branch)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 u[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          frag_t<T> x[NM];
#pragma unroll
          for (int pl = 0; pl < NM; ++pl)
            x[pl] = lds_row8(ox + pl * OPLANE + row_of(ct, c) * PITCH + 32 * ks + 8 * g16);
          u[ks] = mma_planes(tf[ks], x, zero4());
        }
        u[0] += u[1];
        put_opnd<PITCH, OPLANE, NP>(ow, row_of(ct, c), 16 * w + quad_place(g16), u[0] * el);
        if constexpr (GRAD) put_opnd<PITCH, OPLANE, NP>(ov, row_of(ct, c), r4, u[0]);
      }
      const float decay = last;
      if constexpr (kAhead) {
        load_keys(blk + 1, 1);
      } else {
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) load_column(columns, t, ks);
      }
      load_rest(blk + 1);
      lds_barrier();

#pragma unroll
      for (int t = 0; t < TPW; ++t) s[t] *= decay;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        frag_t<T> uf[NP];
#pragma unroll
        for (int pl = 0; pl < NP; ++pl)
          uf[pl] = lds_row8(ow + pl * OPLANE + (32 * cg + col_place(n)) * PITCH + 16 * ks + 8 * h2);
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) s[t] = mma32(kc[t][ks], uf[pl], s[t]);
      }
    }
    if (p.state_out) {
      float* so = p.state_out + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) so[(krow + 32 * t + state_row(i, h2)) * D + vcol] = s[t][i];
    }
  } else if constexpr (GRAD) {
    // the state at the block's start, [dv][dk] in planes
    auto keep_state = [&](int blk) {
      const T* copy = os + (kTwoCopies ? (blk & 1) * COPY : 0);
      T* sn = reinterpret_cast<T*>(p.snap) + slot_of(blk) * (NP * D * D);
#pragma unroll
      for (int pl = 0; pl < NP; ++pl)
        for (int i = tid - 256; i < CS::SL * D / 8; i += 256) {
          const int row = i / (D / 8), at = i % (D / 8) * 8, col = slice * CS::SL + (row & 32) + col_at(row & 31);
          copy8(sn + pl * D * D + (int64_t)col * D + at, copy + pl * CS::SPLANE + row * CS::SPITCH + at);
        }
    };
    for (int blk = 0; blk < nblk; ++blk) {
      lds_barrier();
      if constexpr (!kTwoCopies) keep_state(blk);
      lds_barrier();
      lds_barrier();
      if constexpr (kTwoCopies) keep_state(blk);
      // V' in planes of whole tensors
#pragma unroll
      for (int pl = 0; pl < NP; ++pl) {
        const auto ur = value_rsrc(reinterpret_cast<const T*>(p.u) + pl * (int64_t)p.total * vs, blk);
#pragma unroll
        for (int g = 0; g < CG; ++g) {
          const vec4_t<T> x = *reinterpret_cast<const vec4_t<T>*>(ov + pl * OPLANE + row_of(2 * g, c) * PITCH + r4);
          const vec4_t<T> y = *reinterpret_cast<const vec4_t<T>*>(ov + pl * OPLANE + row_of(2 * g + 1, c) * PITCH + r4);
#pragma unroll
          for (int i = 0; i < 4; ++i) buf_put_pair(ur, pair_off[i] + 32 * g * SZ, (float)x[i], (float)y[i], tag);
        }
      }
    }
  } else {
    frag_t<T> qf[D / 32], mf[2][NM];
#pragma unroll
    for (int pl = 0; pl < NM; ++pl) mf[1][pl] = zero_frag<T>();
    f32x4 eg;
    auto load_queries = [&](int blk) {
      const auto rs = key_rsrc(p.qf, blk);
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) qf[ks] = buf_frag(rs, lane_off, query_frag<D>(w, ks) * SZ, tag);
    };
    auto load_rest = [&](int blk) {
      const auto mr = mat_rsrc(p.m, NM, blk);
#pragma unroll
      for (int pl = 0; pl < NM; ++pl)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          if (ks <= (w >> 1)) mf[ks][pl] = buf_frag(mr, lane_off, mat_frag(pl, w, ks) * SZ, tag);
      eg = buf_f4(vec_rsrc(blk), r4 * 4, 0);
    };
    f32x4 o[CT];
    auto query_state = [&](int blk) {
      const T* copy = os + (kTwoCopies ? (blk & 1) * COPY : 0);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) o[ct] = zero4();
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
            o[ct] = mma(qf[ks], lds_row8(copy + pl * CS::SPLANE + row_of(ct, c) * CS::SPITCH + 32 * ks + 8 * g16), o[ct]);
    };
    load_queries(0);
    load_rest(0);
    for (int blk = 0; blk < nblk; ++blk) {
      lds_barrier();
      if constexpr (!kTwoCopies) query_state(blk);
      lds_barrier();
      const f32x4 in = p.scale * eg;
      lds_barrier();
      if constexpr (kTwoCopies) query_state(blk);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        o[ct] *= in;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          frag_t<T> x[NM];
#pragma unroll
          for (int pl = 0; pl < NM; ++pl) x[pl] = lds_row8(ox + pl * OPLANE + row_of(ct, c) * PITCH + 32 * ks + 8 * g16);
          o[ct] = mma_planes(mf[ks], x, o[ct]);
        }
      }
      const auto orsrc = value_rsrc(p.o, blk);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < CG; ++g) buf_put_pair(orsrc, pair_off[i] + 32 * g * SZ, o[2 * g][i], o[2 * g + 1][i], tag);
      load_queries(blk + 1);
      load_rest(blk + 1);
    }
  }
}

template <typename T, int D, bool GRAD>
static hipError_t launch_forward(const DeltaParams& p, hipStream_t stream) {
  using CS = ChainShape<T, D>;
  hipLaunchKernelGGL((delta_prep_kernel<T, D, GRAD>), dim3(p.batch * p.blocks_max, p.k_heads), dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_chain_kernel<T, D, GRAD>), dim3(CS::NSL * p.batch * p.heads), dim3(512), 0, stream, p);
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

template <typename T>
static void plane_layout(DeltaLayout& l) {
  l.planes = Planes<T>::N;
  l.mat_planes = MatPlanes<T, true>::N;
  l.mat_plane = kB * kB * sizeof(T);
}

DeltaLayout delta_layout(int batch, int seqlen, int dtype, bool packed, int total) {
  DeltaLayout l;
  const size_t per = ((size_t)seqlen + kB - 1) / kB;
  l.blocks = packed ? (size_t)total / kB + batch : per * batch;
  if (dtype == 1)
    plane_layout<bf16>(l);
  else
    plane_layout<float>(l);
  return l;
}

}  // namespace ret
