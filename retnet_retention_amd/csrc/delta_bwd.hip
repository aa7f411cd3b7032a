// Gradients of the gated delta rule's chunkwise form. The forward's walk is
// run again (delta_fwd.hip, which keeps V', the state at each block's start and
// the row sums o . dO); then, with dS+ the gradient of a block's final state,
//     dV' = e^(G_last - G) K dS+ + P^T dO,   dv = T^T dV'  (X = V - e^G K S),
//     dS = e^(G_last) dS+ + Q^T (scale e^G dO) - K^T (e^G dv)
// goes through the blocks from the last to the first (delta_reverse_kernel),
// and per block, with all of the above at hand (delta_qk_grad_kernel),
//     dP = (dO V'^T) scale E  (s <= r),   dA = -(dv V'^T) E  (s < r),
//     dq = scale e^G dO S^T + dP K,
//     dk = e^(G_last - G) V' dS+^T - e^G dv S^T + dP^T Q + (dA + dA^T) K.
// The decays and strengths take row sums only. Scaling the state's history up
// to token t by a factor is the same as scaling every later output and
// dividing every later value by it, so with d_t = o_t . dO_t - v_t . dv_t
//     d log_decay_t = sum over t' >= t of d_t' + <S_end, dS_end>,
// summed inside groups of kDeltaGroup blocks from the product of the state and
// its gradient at the group's end (a sum over a whole sequence would cancel);
//     d beta_t = dv_t . V'_t / beta_t^2   (V' is beta times the prediction error,
//     dv beta times what the write of it gains).
#include "delta_common.hpp"

namespace ret {

hipError_t launch_delta_forward(const DeltaParams& p, int d, int dtype, bool grad, hipStream_t stream);

// The gradient of the state, from a sequence's last block to its first: the
// same division of work and the same three exchanges as delta_chain_kernel.
// The second four waves form P^T dO, put scale e^G dO where the state waves
// read it, and take the row sums. 333 us for 4 sequences of 32 blocks, 10 heads
// of 256 (320 workgroups on 256 CUs: two rounds, the second a quarter full), and
// the forward's walk before it 335; 171 and 193 us for 63 blocks, 16 heads of
// 128 (64 workgroups, 2.7 us a block). With 128 registers a lane, for two
// workgroups a CU at 128, both spill: 720 us for a backward that took 407.
template <typename T, int D>
__global__ __launch_bounds__(512) void delta_reverse_kernel(DeltaParams p) {
  using CS = ChainShape<T, D>;
  constexpr int NP = Planes<T>::N, NM = MatPlanes<T, true>::N, SZ = sizeof(T);
  constexpr int RG = CS::RG, TPW = CS::TPW, CT = CS::CT, CG = CS::CG, PITCH = CS::PITCH, OPLANE = CS::OPLANE;
  constexpr bool kAhead = SZ == 2;  // fp32 keys do not fit the registers a block ahead
  T* const tag = nullptr;
  __shared__ __attribute__((aligned(16))) f32x4 part[4 * 512];
  __shared__ __attribute__((aligned(16))) f32x4 quarter[16 * CT * 16];
  __shared__ __attribute__((aligned(16))) T od[OPLANE], oq[CS::OPND], ox[OPLANE * NM], ow[CS::OPND];

  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_i(tid >> 6), w = wave & 3;
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int slice = id % CS::NSL, bh = id / CS::NSL, h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.k_heads);
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  const int r4 = 16 * w + 4 * g16;
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  const int nblk = (len + kB - 1) / kB;
  const int64_t vs = (int64_t)p.heads * D;
  const uint32_t vrow = (uint32_t)vs * SZ;
  // descriptors of block blk (no rows: nothing is read)
  auto rows_of = [&](int blk) { return blk >= 0 ? min(kB, len - blk * kB) : 0; };
  auto key_rsrc = [&](const void* x, int blk) {  // keys or queries in the lanes' order
    return scalar_rsrc(reinterpret_cast<const T*>(x) + ((int64_t)(base + blk) * p.k_heads + hk) * (kB * D),
                       blk >= 0 ? kB * D * SZ : 0);
  };
  auto value_rsrc = [&](const void* x, int blk) {
    return scalar_rsrc(reinterpret_cast<const T*>(x) + (tok0 + (int64_t)blk * kB) * vs + h * D, rows_of(blk) * vrow);
  };
  auto slot_of = [&](int blk) { return (int64_t)(base + blk) * p.heads + h; };
  auto mat_rsrc = [&](const void* x, int blk) {
    return scalar_rsrc(reinterpret_cast<const T*>(x) + slot_of(blk) * (NM * kB * kB), blk >= 0 ? NM * kB * kB * SZ : 0);
  };
  auto vec_rsrc = [&](int blk) { return scalar_rsrc(p.vec + slot_of(blk) * (4 * kB), blk >= 0 ? 4 * kB * 4 : 0); };
  const uint32_t lane_off = 8 * lane * SZ;
  uint32_t pair_off[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pair_off[i] = (r4 + i) * vrow + (slice * CS::SL + 2 * c) * SZ;
  const int krow = CS::KR * (w % RG), cg = w / RG, vcol = slice * CS::SL + 32 * cg + n;
  auto load_mat = [&](frag_t<T>(&f)[2][NM], const void* x, int blk) {
    const auto rs = mat_rsrc(x, blk);
#pragma unroll
    for (int pl = 0; pl < NM; ++pl)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks >= (w >> 1)) f[ks][pl] = buf_frag(rs, lane_off, mat_frag(pl, w, ks) * SZ, tag);  // upper triangular
  };
  auto load_keys = [&](frag_t<T>(&f)[2][CS::KS], int blk) {
    const auto rs = key_rsrc(p.kf, blk);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int ks = 0; ks < CS::KS; ++ks)
        f[rt][ks] = buf_frag(rs, lane_off, key_frag(krow / 16 + ks, rt) * SZ, tag);
  };
  auto load_column = [&](frag_t<T>(&f)[TPW][4], __amdgpu_buffer_rsrc_t rs, int t, int ks) {
    f[t][ks] = buf_frag(rs, lane_off, column_frag(krow / 32 + t, ks) * SZ, tag);
  };
  auto load_columns = [&](frag_t<T>(&f)[TPW][4], const void* x, int blk) {
    const auto rs = key_rsrc(x, blk);
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) load_column(f, rs, t, ks);
  };
  auto load_pairs = [&](PairOf<T>(&x)[CG][4], const void* from, int blk) {
    const auto rs = value_rsrc(from, blk);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < CG; ++g) x[g][i] = buf_pair(rs, pair_off[i] + 32 * g * SZ, tag);
  };
  // each quarter's P^T dO on its way to the state wave, then its dv back
  f32x4* my_quarter = quarter + (4 * w + g16) * (CT * 16) + c;

  if (wave < 4) {
    f32x16 s[TPW];
#pragma unroll
    for (int t = 0; t < TPW; ++t) s[t] = zero16();
    if (p.d_state_out) {
      const float* si = p.d_state_out + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = si[(krow + 32 * t + state_row(i, h2)) * D + vcol];
    }
    frag_t<T> kf[2][CS::KS], kc[TPW][4], qc[TPW][4], tf[2][NM];
#pragma unroll
    for (int pl = 0; pl < NM; ++pl) tf[0][pl] = zero_frag<T>();
    f32x4 eg, el;
    float last;
    auto load_rest = [&](int blk) {
      load_mat(tf, p.tt, blk);
      const auto er = vec_rsrc(blk);
      eg = buf_f4(er, r4 * 4, 0);
      el = buf_f4(er, r4 * 4, kB * 4);
      last = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(er, 0, (kB - 1) * 4, 0));
    };
    load_rest(nblk - 1);
    if constexpr (kAhead) {
      load_keys(kf, nblk - 1);
      load_columns(kc, p.kc, nblk - 1);
    }
    lds_barrier();

    for (int blk = nblk - 1; blk >= 0; --blk) {
      const int64_t slot = slot_of(blk);
      const bool group_end = (blk + 1) % kDeltaGroup == 0 || blk == nblk - 1;
      if (group_end && (blk != nblk - 1 || p.d_state_out)) {
        // <state, its gradient> at the group's end, this wave's part
        const int64_t at =
            (((int64_t)(base / kDeltaGroup + b + blk / kDeltaGroup) * p.heads + h) * CS::NSL + slice) * 4 + w;
        const float* an = p.anchor + at * (TPW * 1024) + lane * 4;
        float dot = 0.f;
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(an + (4 * t + q) * 256);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += x[i] * s[t][4 * q + i];
          }
        dot = sum64(dot);
        if (lane == 0) p.adot[at] = dot;
      }
      if constexpr (!kAhead) load_keys(kf, blk);
      const auto queries = key_rsrc(p.qc, blk);
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
            load_column(qc, queries, t, 2 * SLI);
            load_column(qc, queries, t, 2 * SLI + 1);
          }
          T* sn = reinterpret_cast<T*>(p.dsnap) + (slot * D + vcol) * D + krow + 16 * ks + 8 * h2;
          *reinterpret_cast<frag_t<T>*>(sn) = f[ks].f[0];
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

      // dV' of the quarter (zero behind the sequence's end: K and dO are)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        put_opnd<PITCH, OPLANE, NM>(ox, row_of(ct, c), r4,
                                    get_partial<RG>(part, ct, 4 * w + g16, c) * el + my_quarter[16 * ct]);
      if constexpr (kAhead) load_keys(kf, blk - 1);
      lds_barrier();

      // dv = T^T dV'; the state takes -e^G dv
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 dv[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          frag_t<T> x[NM];
#pragma unroll
          for (int pl = 0; pl < NM; ++pl)
            x[pl] = lds_row8(ox + pl * OPLANE + row_of(ct, c) * PITCH + 32 * ks + 8 * g16);
          dv[ks] = mma_planes(tf[ks], x, zero4());
        }
        dv[0] += dv[1];
        put_opnd<PITCH, OPLANE, NP>(ow, row_of(ct, c), 16 * w + quad_place(g16), -eg * dv[0]);
        my_quarter[16 * ct] = dv[0];
      }
      const float decay = last;
      load_rest(blk - 1);
      lds_barrier();
      auto add = [&](const frag_t<T>(&f)[TPW][4], const T* opnd) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          frag_t<T> x[NP];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
            x[pl] = lds_row8(opnd + pl * OPLANE + (32 * cg + col_place(n)) * PITCH + 16 * ks + 8 * h2);
#pragma unroll
          for (int t = 0; t < TPW; ++t)
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) s[t] = mma32(f[t][ks], x[pl], s[t]);
        }
      };
#pragma unroll
      for (int t = 0; t < TPW; ++t) s[t] *= decay;
      if constexpr (!kAhead) load_columns(qc, p.qc, blk);
      add(qc, oq);
      if constexpr (!kAhead) load_columns(kc, p.kc, blk);
      add(kc, ow);
      if constexpr (kAhead) load_columns(kc, p.kc, blk - 1);
    }
    if (p.d_state_in) {
      float* so = p.d_state_in + (int64_t)bh * D * D;
#pragma unroll
      for (int t = 0; t < TPW; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) so[(krow + 32 * t + state_row(i, h2)) * D + vcol] = s[t][i];
    }
  } else {
    frag_t<T> pf[2][NM];
#pragma unroll
    for (int pl = 0; pl < NM; ++pl) pf[0][pl] = zero_frag<T>();
    PairOf<T> dout[CG][4], dnext[CG][4], v[CG][4], u[NP][CG][4];
    f32x4 eg;
    auto put_dout = [&](const PairOf<T>(&x)[CG][4]) {  // exact in T
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        vec4_t<T> y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (T)x[ct >> 1][i].get(ct & 1);
        *reinterpret_cast<vec4_t<T>*>(od + row_of(ct, c) * PITCH + r4) = y;
      }
    };
    auto load_values = [&](int blk) {
      load_pairs(v, p.v, blk);
#pragma unroll
      for (int pl = 0; pl < NP; ++pl) load_pairs(u[pl], reinterpret_cast<const T*>(p.u) + pl * (int64_t)p.total * vs, blk);
    };
    load_pairs(dout, p.dout, nblk - 1);
    load_mat(pf, p.pt, nblk - 1);
    eg = buf_f4(vec_rsrc(nblk - 1), r4 * 4, 0);
    load_values(nblk - 1);
    load_pairs(dnext, p.dout, nblk - 2);
    put_dout(dout);
    lds_barrier();
    for (int blk = nblk - 1; blk >= 0; --blk) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 x = zero4();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const frag_t<T> d = lds_row8(od + row_of(ct, c) * PITCH + 32 * ks + 8 * g16);
#pragma unroll
          for (int pl = NM - 1; pl >= 0; --pl) x = mma(pf[ks][pl], d, x);
        }
        my_quarter[16 * ct] = x;
      }
      load_mat(pf, p.pt, blk - 1);
      lds_barrier();
      // scale e^G dO, for the state waves after the third barrier
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p.scale * eg[i] * dout[ct >> 1][i].get(ct & 1);
        put_opnd<PITCH, OPLANE, NP>(oq, row_of(ct, c), 16 * w + quad_place(g16), x);
      }
      put_dout(dnext);
#pragma unroll
      for (int g = 0; g < CG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) dout[g][i] = dnext[g][i];
      load_pairs(dnext, p.dout, blk - 2);
      eg = buf_f4(vec_rsrc(blk - 1), r4 * 4, 0);
      lds_barrier();
      lds_barrier();
      // dv and the row sums of the quarter
      const auto rs = value_rsrc(p.dv, blk);
      f32x4 vdv = zero4(), uv = zero4();
#pragma unroll
      for (int g = 0; g < CG; ++g) {
        f32x4 dv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          dv[e] = my_quarter[16 * (2 * g + e)];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y = 0.f;
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) y += u[pl][g][i].get(e);
            vdv[i] += dv[e][i] * v[g][i].get(e);
            uv[i] += dv[e][i] * y;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) buf_put_pair(rs, pair_off[i] + 32 * g * SZ, dv[0][i], dv[1][i], tag);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vdv[i] = sum16(vdv[i]);
        uv[i] = sum16(uv[i]);
      }
      if (c == 0) {
        *reinterpret_cast<f32x4*>(p.vdv + (slot_of(blk) * CS::NSL + slice) * kB + r4) = vdv;
        *reinterpret_cast<f32x4*>(p.udv + (slot_of(blk) * CS::NSL + slice) * kB + r4) = uv;
      }
      load_values(blk - 1);
    }
  }
}

// d q and d k of one block and key head, summed over the value heads that
// share it (GROUPED: more than one); wave w the key columns 32 w .. + 31. Bound
// by the two states a block reads, D x D each: they pass through LDS by 32 value
// columns, the next tile (two buffers, fp32 one) on its way while one is
// multiplied, and each of dO, dv and V' is read once for all its products. 161
// us for 1280 blocks of 256 x 256 (336 MB of states, 294 MB of rows: 3.9 TB/s);
// 70 us with two value heads of 128 a key head.
// Products of a wave are straight lines of matrix instructions with no branch
// among them. Operands are one bf16 value here (2^-9 each, a sum of independent
// roundings below that of the bf16 result): dq and dk are off by 2.7e-3 and
// 3.0e-3 where their own rounding gives 1.7e-3.
template <typename T, int D, bool GROUPED>
__global__ __launch_bounds__(2 * D) void delta_qk_grad_kernel(DeltaParams p) {
  constexpr int NW = D / 32, TW = 8 / NW;  // tasks of 16 rows of dP and dA a wave
  constexpr int DV = 32;                   // value columns of a state tile in LDS
  constexpr int BUFS = sizeof(T) == 2 ? 2 : 1;
  using ST = LTile<T, DV, D, kColTile>;
  constexpr int PA = sizeof(T) == 2 ? 40 : 36;  // pitch of the row operands
  constexpr int PM = sizeof(T) == 2 ? 72 : 68;  // pitch of the 64 x 64 matrices
  constexpr int ROWS = 3 * kB * PA;
  __shared__ __attribute__((aligned(1024))) char tiles[2 * BUFS * ST::BYTES];
  __shared__ __attribute__((aligned(16))) T row_ops[BUFS * ROWS];  // [dO, dv, V'][64][PA]
  __shared__ __attribute__((aligned(16))) T mp[kB * PM], mpt[kB * PM], ms[kB * PM];
  __shared__ double sg[kB];
  T* const tag = nullptr;

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6);
  const int b = blockIdx.x / p.blocks_max, blk = blockIdx.x % p.blocks_max, hk = blockIdx.y;
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  if (blk * kB >= len) return;
  const int rows = min(kB, len - blk * kB);
  const int64_t row0 = tok0 + blk * kB;
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;
  const int group = GROUPED ? p.heads / p.k_heads : 1;
  // keys and queries by columns, the wave's 32
  const int64_t key_slot = ((int64_t)(base + blk) * p.k_heads + hk) * (kB * D) + 8 * lane;
  const T* KC = reinterpret_cast<const T*>(p.kc) + key_slot;
  const T* QC = reinterpret_cast<const T*>(p.qc) + key_slot;

  f32x16 dq[2] = {zero16(), zero16()}, dk[2] = {zero16(), zero16()};
  for (int hh = 0; hh < group; ++hh) {
    const int h = hk * group + hh;
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    const T* src[3] = {reinterpret_cast<const T*>(p.dout) + row0 * vs + h * D,
                       reinterpret_cast<const T*>(p.dv) + row0 * vs + h * D,
                       reinterpret_cast<const T*>(p.u) + row0 * vs + h * D};
    const T* SN = reinterpret_cast<const T*>(p.snap) + slot * D * D;
    const T* DN = reinterpret_cast<const T*>(p.dsnap) + slot * D * D;
    TileLoads<T, ST, NW> sloads;
    sloads.init(D, lane);
    constexpr int RN = (3 * kB * (DV / 8) + 2 * D - 1) / (2 * D);  // row operands: chunks of 8 a thread
    Raw8<T> raw[RN];
    auto ask = [&](int d0) {
      char* to = tiles + (d0 / DV % BUFS) * 2 * ST::BYTES;
      sloads.issue(to, SN, D, d0, w);
      sloads.issue(to + ST::BYTES, DN, D, d0, w);
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int at = tid + i * 2 * D, m = at / (kB * (DV / 8)), r = at / (DV / 8) % kB, j = at % (DV / 8) * 8;
        raw[i] = Raw8<T>{};
        if (m < 3 && r < rows) raw[i] = ld_raw8((m == 0 ? src[0] : m == 1 ? src[1] : src[2]) + r * vs + d0 + j);
      }
    };
    if constexpr (GROUPED) __syncthreads();  // the last head's reads
    if (w == 0) {
      float g = lane < rows ? p.log_decay[(row0 + lane) * p.heads + h] : 0.f;
      if (g < kMinLogDecay) g = kMinLogDecay;
      double s = g;
#pragma unroll
      for (int o = 1; o < 64; o *= 2) {
        const double y = __shfl_up(s, o, 64);
        if (lane >= o) s += y;
      }
      sg[lane] = s;
    }
    for (int i = tid; i < 3 * kB * PM; i += 2 * D) (i < kB * PM ? mp : i < 2 * kB * PM ? mpt : ms)[i % (kB * PM)] = (T)0.f;

    f32x4 acc[TW][4];
#pragma unroll
    for (int k = 0; k < TW; ++k)
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) acc[k][ct] = zero4();
    // dO S^T, V' dS^T and dv S^T over the value columns
    f32x16 a0[2] = {zero16(), zero16()}, a1[2] = {zero16(), zero16()}, a2[2] = {zero16(), zero16()};
    ask(0);
    for (int d0 = 0; d0 < D; d0 += DV) {
      const char* tile = tiles + (d0 / DV % BUFS) * 2 * ST::BYTES;
      T* ops = row_ops + (d0 / DV % BUFS) * ROWS;
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int at = tid + i * 2 * D, m = at / (kB * (DV / 8)), r = at / (DV / 8) % kB, j = at % (DV / 8) * 8;
        if (m < 3) st_raw8(ops + (m * kB + r) * PA + j, raw[i], true);
      }
      __builtin_amdgcn_s_waitcnt(0);  // the tiles (LDS loads run past the compiler's counting)
      lds_barrier();
      if (BUFS == 2 && d0 + DV < D) ask(d0 + DV);
#pragma unroll
      for (int k = 0; k < TW; ++k) {
        const int task = w + k * NW, rb = task & 3, which = task >> 2;
        const frag_t<T> a = lds_row8(ops + (which * kB + 16 * rb + c) * PA + 8 * g16);
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)  // (all four: the upper ones are left out below)
          acc[k][ct] = mma(a, lds_row8(ops + (2 * kB + 16 * ct + c) * PA + 8 * g16), acc[k][ct]);
      }
#pragma unroll
      for (int ks = 0; ks < DV / 16; ++ks) {
        const frag_t<T> fs = state_tile_col8<ST>(tile, 16 * ks, 32 * w, lane, tag);
        const frag_t<T> fd = state_tile_col8<ST>(tile + ST::BYTES, 16 * ks, 32 * w, lane, tag);
        // the column fragments' order of the contraction
        auto row = [&](int m, int rt) {
          const T* at = ops + (m * kB + 32 * rt + n) * PA + 16 * ks + 4 * h2;
          const vec4_t<T> lo = *reinterpret_cast<const vec4_t<T>*>(at), hi = *reinterpret_cast<const vec4_t<T>*>(at + 8);
          frag_t<T> f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] = lo[j];
            f[4 + j] = hi[j];
          }
          return f;
        };
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          a0[rt] = mma32(row(0, rt), fs, a0[rt]);
          a2[rt] = mma32(row(1, rt), fs, a2[rt]);
          a1[rt] = mma32(row(2, rt), fd, a1[rt]);
        }
      }
      if (BUFS == 1 && d0 + DV < D) {
        lds_barrier();
        ask(d0 + DV);
      }
    }
    frag_t<T> fq[4], fk[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      fq[ks] = *reinterpret_cast<const frag_t<T>*>(QC + column_frag(w, ks));
      fk[ks] = *reinterpret_cast<const frag_t<T>*>(KC + column_frag(w, ks));
    }
    // dP (both ways round) and dA + dA^T
#pragma unroll
    for (int k = 0; k < TW; ++k) {
      const int task = w + k * NW, rb = task & 3, which = task >> 2;
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        const int s = 16 * ct + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * rb + 4 * g16 + i;
          const float e = s <= r ? __builtin_amdgcn_exp2f((float)((sg[r] - sg[s]) * 1.4426950408889634)) : 0.f;
          if (which == 0 && s <= r) {
            const T x = (T)(p.scale * e * acc[k][ct][i]);
            mp[r * PM + s] = x;
            mpt[s * PM + r] = x;
          }
          if (which == 1 && s < r) {
            const T x = (T)(-e * acc[k][ct][i]);
            ms[r * PM + s] = x;
            ms[s * PM + r] = x;
          }
        }
      }
    }
    const float* vec = p.vec + slot * (4 * kB);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 eg = *reinterpret_cast<const f32x4*>(vec + 32 * rt + 8 * q + 4 * h2);
        const f32x4 el = *reinterpret_cast<const f32x4*>(vec + kB + 32 * rt + 8 * q + 4 * h2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = p.scale * eg[i] * a0[rt][4 * q + i];
          const float y = el[i] * a1[rt][4 * q + i] - eg[i] * a2[rt][4 * q + i];
          dq[rt][4 * q + i] = GROUPED ? dq[rt][4 * q + i] + x : x;
          dk[rt][4 * q + i] = GROUPED ? dk[rt][4 * q + i] + y : y;
        }
      }
    __syncthreads();
    // dP^T Q, dP K and (dA + dA^T) K
    auto mrow = [&](const T* m, int rt, int ks) {
      const T* at = m + (32 * rt + n) * PM + 16 * ks + 4 * h2;
      const vec4_t<T> lo = *reinterpret_cast<const vec4_t<T>*>(at), hi = *reinterpret_cast<const vec4_t<T>*>(at + 8);
      frag_t<T> f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = lo[j];
        f[4 + j] = hi[j];
      }
      return f;
    };
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        dk[rt] = mma32(mrow(mpt, rt, ks), fq[ks], dk[rt]);
        dq[rt] = mma32(mrow(mp, rt, ks), fk[ks], dq[rt]);
        dk[rt] = mma32(mrow(ms, rt, ks), fk[ks], dk[rt]);
      }
  }
  T* DQ = reinterpret_cast<T*>(p.dq) + row0 * qs + hk * D + 32 * w + state_col(n);
  T* DK = reinterpret_cast<T*>(p.dk) + row0 * qs + hk * D + 32 * w + state_col(n);
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 32 * rt + 8 * (i / 4) + 4 * h2 + i % 4;
      if (r < rows) {
        DQ[r * qs] = (T)dq[rt][i];
        DK[r * qs] = (T)dk[rt][i];
      }
    }
}

// d log decay and d beta from the row sums, one wave per (group of blocks,
// head): 14 us for 640 groups, the latency of its loads.
__global__ __launch_bounds__(64) void delta_gate_grad_kernel(DeltaParams p, int slices) {
  const int groups = (p.blocks_max + kDeltaGroup - 1) / kDeltaGroup;
  const int b = blockIdx.x / groups, grp = blockIdx.x % groups, h = blockIdx.y, lane = threadIdx.x;
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  const int nblk = (len + kB - 1) / kB;
  if (grp * kDeltaGroup >= nblk) return;
  const int last = min(nblk, (grp + 1) * kDeltaGroup) - 1;
  float carry = 0.f;
  if (last != nblk - 1 || p.d_state_out) {
    const float* ad = p.adot + ((int64_t)(base / kDeltaGroup + b + grp) * p.heads + h) * slices * 4;
    for (int i = 0; i < slices * 4; ++i) carry += ad[i];
  }
  for (int blk = last; blk >= grp * kDeltaGroup; --blk) {
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    float d = 0.f, x = 0.f;
    for (int s = 0; s < slices; ++s) {
      const int64_t at = (slot * slices + s) * kB + lane;
      d += p.odo[at] - p.vdv[at];
      x += p.udv[at];
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const float y = __shfl_down(d, o, 64);
      if (lane + o < 64) d += y;
    }
    d += carry;
    carry = __shfl(d, 0, 64);
    const int r = blk * kB + lane;
    if (r < len) {
      const int64_t at = (tok0 + r) * p.heads + h;
      // The gradient is the factor exp(log decay) times what the state before it
      // gives: zero where that is zero. The sum would be its own rounding there.
      const bool none = (r == 0 && !p.state_in) || p.log_decay[at] < kZeroLogDecay;
      p.d_log_decay[at] = none ? 0.f : d;
      const float beta = p.vec[slot * (4 * kB) + 2 * kB + lane];
      p.d_beta[at] = x / beta / beta;
    }
  }
}

template <typename T, int D>
static hipError_t launch_backward(const DeltaParams& p, hipStream_t stream) {
  using CS = ChainShape<T, D>;
  hipLaunchKernelGGL((delta_reverse_kernel<T, D>), dim3(CS::NSL * p.batch * p.heads), dim3(512), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(p.batch * p.blocks_max, p.k_heads);
  if (p.heads == p.k_heads)
    hipLaunchKernelGGL((delta_qk_grad_kernel<T, D, false>), grid, dim3(2 * D), 0, stream, p);
  else
    hipLaunchKernelGGL((delta_qk_grad_kernel<T, D, true>), grid, dim3(2 * D), 0, stream, p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int groups = (p.blocks_max + kDeltaGroup - 1) / kDeltaGroup;
  hipLaunchKernelGGL(delta_gate_grad_kernel, dim3(p.batch * groups, p.heads), dim3(64), 0, stream, p, CS::NSL);
  return hipGetLastError();
}

hipError_t launch_delta_bwd(const DeltaParams& p, int d, int dtype, hipStream_t stream) {
  const hipError_t e = launch_delta_forward(p, d, dtype, true, stream);
  if (e != hipSuccess) return e;
  if (dtype == 1) {
    switch (d) {
      case 64: return launch_backward<bf16, 64>(p, stream);
      case 128: return launch_backward<bf16, 128>(p, stream);
      case 256: return launch_backward<bf16, 256>(p, stream);
    }
  } else {
    switch (d) {
      case 64: return launch_backward<float, 64>(p, stream);
      case 128: return launch_backward<float, 128>(p, stream);
      case 256: return launch_backward<float, 256>(p, stream);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace ret
