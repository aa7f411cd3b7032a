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

// The state's way through one sequence's blocks, for SL value columns of one
// head; GRAD: the same walk for the backward, which keeps V', the states and
// the row sums o . dO in place of the output.
// Bound by the way from one block's state to the next, which takes three
// exchanges between the four state waves: each multiplies its key rows of S
// into K S (partial sums of all 64 tokens); a quarter of the tokens each, they
// add these up to X; V' = T X, a quarter each; then every wave adds K^T V' to
// its rows. The other four waves follow with the output, a quarter of the
// tokens each: Q S from a copy of the state in LDS while the state waves are at
// X and V', then P V'. What a block reads is asked for a block ahead.
template <typename T, int D, bool GRAD>
__global__ __launch_bounds__(512) void delta_chain_kernel(DeltaParams p) {
  using CS = ChainShape<T, D>;
  using KT = KeyTile<T, CS::KR>;
  constexpr int NP = Planes<T>::N, PP = GRAD ? NP : 1, SZ = sizeof(T);
  constexpr int RG = CS::RG, TPW = CS::TPW, CT = CS::CT, CG = CS::CG, PITCH = CS::PITCH, OPLANE = CS::OPLANE;
  T* const tag = nullptr;
  __shared__ __attribute__((aligned(16))) char kt[4 * KT::BYTES];
  __shared__ __attribute__((aligned(16))) f32x4 part[4 * 512];
  __shared__ __attribute__((aligned(16))) T ox[CS::OPND], ov[CS::OPND], ow[CS::OPND];
  __shared__ __attribute__((aligned(16))) T os[CS::SPLANE * PP];

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
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;
  const uint32_t qrow = (uint32_t)qs * SZ, vrow = (uint32_t)vs * SZ;
  // descriptors of block blk (no rows: nothing is read)
  auto rows_of = [&](int blk) { return blk < nblk ? min(kB, len - blk * kB) : 0; };
  auto key_rsrc = [&](const void* x, int blk) {
    return scalar_rsrc(reinterpret_cast<const T*>(x) + (tok0 + (int64_t)blk * kB) * qs + hk * D, rows_of(blk) * qrow);
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
  const uint32_t mat_off = ((16 * w + c) * kB + 8 * g16) * SZ;
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
    if (p.state_in) {
      const float* si = p.state_in + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = si[(krow + 32 * t + state_row(i, h2)) * D + vcol];
    }
    char* my_kt = kt + w * KT::BYTES;
    const uint32_t key_off[2] = {n * qrow + (krow + 8 * h2) * SZ, (32 + n) * qrow + (krow + 8 * h2) * SZ};
    T* my_os = os + (32 * cg + col_place(n)) * CS::SPITCH + krow + 8 * h2;

    frag_t<T> kf[2][CS::KS], tf[NP][2];
    PairOf<T> v[CG][4];
    f32x4 eg, el, beta;
    float last;
    auto load_keys = [&](int blk) {
      const auto rs = key_rsrc(p.k, blk);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ks = 0; ks < CS::KS; ++ks) kf[rt][ks] = buf_frag(rs, key_off[rt] + 16 * ks * SZ, tag);
    };
    auto load_rest = [&](int blk) {
      const auto tr = mat_rsrc(p.t, NP, blk);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > (w >> 1)) break;  // T is lower triangular
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) tf[pl][ks] = buf_frag(tr, mat_off + (pl * kB * kB + 32 * ks) * SZ, tag);
      }
      const auto vr = value_rsrc(p.v, blk);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int g = 0; g < CG; ++g) v[g][i] = buf_pair(vr, pair_off[i] + 32 * g * SZ, tag);
      const auto er = vec_rsrc(blk);
      eg = buf_f4(er, r4 * 4);
      el = buf_f4(er, (kB + r4) * 4);
      beta = buf_f4(er, (2 * kB + r4) * 4);
      last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(er, (kB - 1) * 4, 0, 0));
    };
    load_keys(0);
    load_rest(0);

    for (int blk = 0; blk < nblk; ++blk) {
      const int rows = min(kB, len - blk * kB);
      f32x16 ksum[2] = {zero16(), zero16()};
#pragma unroll
      for (int t = 0; t < TPW; ++t)
        static_for<2>([&](auto sl) {
          constexpr int SLI = decltype(sl)::value;
          const Split<T> f = split_acc<SLI>(s[t], tag);
          const int ks = 2 * t + SLI;
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) ksum[rt] = mma32(kf[rt][ks], f.f[pl], ksum[rt]);
#pragma unroll
          for (int pl = 0; pl < PP; ++pl)
            *reinterpret_cast<frag_t<T>*>(my_os + pl * CS::SPLANE + 16 * ks) = f.f[pl];
        });
      put_partial(part, w, ksum, lane);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ks = 0; ks < CS::KS; ++ks) KT::put(my_kt, 32 * rt + n, 16 * ks + 8 * h2, kf[rt][ks]);
      load_keys(blk + 1);
      if constexpr (GRAD) {
        if (blk && blk % kDeltaGroup == 0) {
          float* an = p.anchor + ((((int64_t)(base / kDeltaGroup + b + blk / kDeltaGroup - 1) * p.heads + h) * CS::NSL +
                                   slice) * 4 + w) * (TPW * 1024) + lane * 4;
#pragma unroll
          for (int t = 0; t < TPW; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<f32x4*>(an + (4 * t + q) * 256) =
                  f32x4{s[t][4 * q], s[t][4 * q + 1], s[t][4 * q + 2], s[t][4 * q + 3]};
        }
      }
      lds_barrier();

      // X of the quarter
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const f32x4 ks = get_partial<RG>(part, ct, 4 * w + g16, c);
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = beta[i] * (v[ct >> 1][i].get(ct & 1) - eg[i] * ks[i]);
          x[i] = r4 + i < rows ? y : 0.f;
        }
        put_opnd<PITCH, OPLANE>(ox, 16 * ct + c, r4, x);
      }
      lds_barrier();

      // V' = T X
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 u = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (ks > (w >> 1)) break;
          frag_t<T> a[NP], x[NP];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) {
            a[pl] = tf[pl][ks];
            x[pl] = lds_row8(ox + pl * OPLANE + (16 * ct + c) * PITCH + 32 * ks + 8 * g16);
          }
          u = mma_split2(a, x, u, tag);
        }
        put_opnd<PITCH, OPLANE>(ow, 16 * ct + c, 16 * w + quad_place(g16), u * el);
        put_opnd<PITCH, OPLANE>(ov, 16 * ct + c, r4, u);
      }
      const float decay = last;
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
        for (int t = 0; t < TPW; ++t) {
          const frag_t<T> a = KT::col(my_kt, 16 * ks, 32 * t, lane);
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) s[t] = mma32(a, uf[pl], s[t]);
        }
      }
    }
    if (p.state_out) {
      float* so = p.state_out + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) so[(krow + 32 * t + state_row(i, h2)) * D + vcol] = s[t][i];
    }
    if constexpr (GRAD) {
      if (nblk && p.d_state_out) {  // the last group's copy: only a gradient of the final state meets it
        float* an = p.anchor + ((((int64_t)(base / kDeltaGroup + b + (nblk - 1) / kDeltaGroup) * p.heads + h) * CS::NSL +
                                 slice) * 4 + w) * (TPW * 1024) + lane * 4;
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(an + (4 * t + q) * 256) =
                f32x4{s[t][4 * q], s[t][4 * q + 1], s[t][4 * q + 2], s[t][4 * q + 3]};
      }
    }
  } else {
    frag_t<T> qf[D / 32], pf[PP][2];
    PairOf<T> dout[CG][4];
    f32x4 eg;
    auto load_queries = [&](int blk) {
      const auto rs = key_rsrc(p.q, blk);
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) qf[ks] = buf_frag(rs, (16 * w + c) * qrow + (32 * ks + 8 * g16) * SZ, tag);
    };
    auto load_rest = [&](int blk) {
      const auto pr = mat_rsrc(p.p, PP, blk);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > (w >> 1)) break;
#pragma unroll
        for (int pl = 0; pl < PP; ++pl) pf[pl][ks] = buf_frag(pr, mat_off + (pl * kB * kB + 32 * ks) * SZ, tag);
      }
      eg = buf_f4(vec_rsrc(blk), r4 * 4);
      if constexpr (GRAD) {
        const auto dr = value_rsrc(p.dout, blk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 0; g < CG; ++g) dout[g][i] = buf_pair(dr, pair_off[i] + 32 * g * SZ, tag);
      }
    };
    load_queries(0);
    load_rest(0);
    for (int blk = 0; blk < nblk; ++blk) {
      lds_barrier();
      f32x4 o[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) o[ct] = zero4();
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int pl = 0; pl < PP; ++pl)
            o[ct] = mma(qf[ks], lds_row8(os + pl * CS::SPLANE + (16 * ct + c) * CS::SPITCH + 32 * ks + 8 * g16), o[ct]);
      load_queries(blk + 1);
      if constexpr (GRAD) {
        // the state at the block's start, [dv][dk], for the gradients of q and k
        T* sn = reinterpret_cast<T*>(p.snap) + slot_of(blk) * D * D;
        for (int i = tid - 256; i < CS::SL * D / 8; i += 256) {
          const int row = i / (D / 8), at = i % (D / 8) * 8, pl = row & 31;
          const int col = slice * CS::SL + (row & 32) + 2 * (pl & 15) + (pl >> 4);
          copy8(sn + (int64_t)col * D + at, os + row * CS::SPITCH + at);
        }
      }
      lds_barrier();
      lds_barrier();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        o[ct] *= p.scale * eg;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          if (ks > (w >> 1)) break;
          frag_t<T> u[NP];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) u[pl] = lds_row8(ov + pl * OPLANE + (16 * ct + c) * PITCH + 32 * ks + 8 * g16);
          if constexpr (GRAD) {
            frag_t<T> a[NP];
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) a[pl] = pf[pl][ks];
            o[ct] = mma_split2(a, u, o[ct], tag);
          } else {
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) o[ct] = mma(pf[0][ks], u[pl], o[ct]);
          }
        }
      }
      if constexpr (!GRAD) {
        const auto orsrc = value_rsrc(p.o, blk);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int g = 0; g < CG; ++g)
            buf_put_pair(orsrc, pair_off[i] + 32 * g * SZ, o[2 * g][i], o[2 * g + 1][i], tag);
      } else {
        f32x4 dot = zero4();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) dot[i] += o[ct][i] * dout[ct >> 1][i].get(ct & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) dot[i] = sum16(dot[i]);
        if (c == 0) *reinterpret_cast<f32x4*>(p.odo + (slot_of(blk) * CS::NSL + slice) * kB + r4) = dot;
        // V' in planes of whole tensors
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
          const auto ur = value_rsrc(reinterpret_cast<const T*>(p.u) + pl * (int64_t)p.total * vs, blk);
#pragma unroll
          for (int g = 0; g < CG; ++g) {
            const vec4_t<T> x = *reinterpret_cast<const vec4_t<T>*>(ov + pl * OPLANE + (32 * g + c) * PITCH + r4);
            const vec4_t<T> y = *reinterpret_cast<const vec4_t<T>*>(ov + pl * OPLANE + (32 * g + 16 + c) * PITCH + r4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              buf_put_pair(ur, pair_off[i] + 32 * g * SZ, (float)x[i], (float)y[i], tag);
          }
        }
      }
      load_rest(blk + 1);
    }
  }
}

template <typename T, int D, bool GRAD>
static hipError_t launch_forward(const DeltaParams& p, hipStream_t stream) {
  using CS = ChainShape<T, D>;
  hipLaunchKernelGGL((delta_prep_kernel<T, D, GRAD>), dim3(p.batch * p.blocks_max, p.heads), dim3(256), 0, stream, p);
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
