// Gradients of the gated delta rule's chunkwise form. The forward's walk is
// run again (delta_fwd.hip, which keeps V' and the state at each block's start);
// then, with dS+ the gradient of a block's final state,
//     dV' = e^(G_last - G) K dS+ + P^T dO,   dv = T^T dV'  (X = V - e^G K S),
//     dS = e^(G_last) dS+ + Q^T (scale e^G dO) - K^T (e^G dv)
// goes through the blocks from the last to the first (delta_reverse_kernel),
// and per block, with all of the above at hand (delta_qk_grad_kernel),
//     dP = (dO V'^T) scale E  (s <= r),   dA = -(dv V'^T) E  (s < r),
//     dq = scale e^G dO S^T + dP K,
//     dk = e^(G_last - G) V' dS+^T - e^G dv S^T + dP^T Q + (dA + dA^T) K.
// A log decay stands in every factor E and e^G that crosses its token, so
//     d log_decay_t = sum over s < t <= r of W_rs + sum over r >= t of x_r
//                     + sum over s < t of y_s + e^(G_last) <S, dS+>,
//     W_rs = dP_rs (q_r . k_s) + dA_rs (k_r . k_s),
//     x_r = q_r . (scale e^G dO S^T)_r - k_r . (e^G dv S^T)_r,
//     y_s = k_s . (e^(G_last - G) V' dS+^T)_s,
// each term with that factor. (The difference of row sums o . dO - v . dv gives
// the same value, but terms without the factor cancel in it and leave their
// roundings: where a token forgets much, more than the gradient itself.)
//     d beta_t = dv_t . V'_t / beta_t^2   (V' is beta times the prediction error,
//     dv beta times what the write of it gains).
#include "delta_common.hpp"

namespace ret {

hipError_t launch_delta_forward(const DeltaParams& p, int d, int dtype, bool grad, hipStream_t stream);

// The gradient of the state, from a sequence's last block to its first: the
// same division of work and the same three exchanges as delta_chain_kernel.
// The second four waves form P^T dO, put scale e^G dO where the state waves
// read it, and write dv. 346 us for 4 sequences of 32 blocks, 10 heads
// of 256 (320 workgroups on 256 CUs: two rounds, the second a quarter full), and
// the forward's walk before it 235; 167 and 129 us for 63 blocks, 16 heads of
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
          T* sn = reinterpret_cast<T*>(p.dsnap) + (slot * NP * D + vcol) * D + krow + 16 * ks + 8 * h2;
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<frag_t<T>*>(sn + pl * D * D) = f[ks].f[pl];
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
    PairOf<T> dout[CG][4], dnext[CG][4];
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
    load_pairs(dout, p.dout, nblk - 1);
    load_mat(pf, p.pt, nblk - 1);
    eg = buf_f4(vec_rsrc(nblk - 1), r4 * 4, 0);
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
      // dv of the quarter, and what its type leaves of it
      const auto rs = value_rsrc(p.dv, blk);
#pragma unroll
      for (int g = 0; g < CG; ++g) {
        const f32x4 x = my_quarter[16 * (2 * g)], y = my_quarter[16 * (2 * g + 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) buf_put_pair(rs, pair_off[i] + 32 * g * SZ, x[i], y[i], tag);
        if constexpr (NP > 1) {
          const auto rest = value_rsrc(p.dv_rest, blk);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            buf_put_pair(rest, pair_off[i] + 32 * g * SZ, x[i] - (float)(T)x[i], y[i] - (float)(T)y[i], tag);
        }
      }
    }
  }
}

// sum of a_j b_j over a fragment's elements
__device__ __forceinline__ float dot_frag(const bf16x8& a, const bf16x8& b, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    c = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a[j], a[j + 1]}, bf16x2{b[j], b[j + 1]}, c, false);
  return c;
}
__device__ __forceinline__ float dot_frag(const f32x8& a, const f32x8& b, float c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = fmaf(a[j], b[j], c);
  return c;
}

// Sum over the lanes up to this one. Only lower lanes are added, so a lane's sum
// takes no rounding from what it leaves out.
__device__ __forceinline__ float scan64(float x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const float y = __shfl_up(x, o, 64);
    x += lane >= o ? y : 0.f;
  }
  return x;
}

// Gradients of one block and key head: dq and dk, summed over the value heads
// that share it (GROUPED: more than one), and each value head's d log decay and
// d beta. Wave w takes the key columns 32 w .. + 31. The two states of a block
// pass through LDS by 16 value columns, the next ones on their way while some are
// multiplied; each of dO, dv and V' is read once for all its products. States,
// dv and V' come as their planes (bf16: two values, so that dq and dk are at
// their own rounding and the decays' gradients good to a few 1e-6).
// A log decay's gradient is the sum of every term that its factor stands in:
// weights between tokens on both sides of it (w: the products of dP with Q K^T and
// of dA with K K^T), what later tokens read of the state before the block (x),
// what earlier ones leave in the state after it (y), and what passes through the
// block (z). Nothing cancels that lacks the factor, so the error carries it too.
// Bound by memory while the states pass (two thirds of a block's 49 us: 42 KB a
// step of 2.1 us on each of 256 CUs), then by one workgroup a CU working alone on
// what follows: 297 us for 1280 blocks of 256 x 256 (671 MB of states, 210 MB of
// rows). One bf16 value a state took 161 and left dq 2.9e-3 and dk 3.2e-3 off (now
// 1.7e-3, their own rounding). 124 us with two value heads of 128 a key head.
// Shared key heads keep dq and dk beside the sums of a head: 39 (bf16) and 74
// (fp32) vector registers of a lane spill at 256, 30 and 42 at 64, written and read
// once a value head; fp32 at 128 without sharing spills 4 for two workgroups a CU.
// Products of a wave are straight lines of matrix instructions with no branch
// among them.
template <typename T, int D, bool GROUPED>
__global__ __launch_bounds__(2 * D, D > 64 && !GROUPED ? 2 : 1) void delta_qk_grad_kernel(DeltaParams p) {
  constexpr int NP = Planes<T>::N, SZ = sizeof(T);
  constexpr int NW = D / 32, TW = 8 / NW;  // 32 x 32 tiles of dP and dA a wave
  constexpr int DV = 16;                   // value columns of a state tile in LDS
  using ST = LTile<T, DV, D, kColTile>;
  constexpr int PA = SZ == 2 ? 24 : 20;  // pitch of the row operands
  constexpr int PM = SZ == 2 ? 72 : 68;  // pitch of the 64 x 64 operands
  constexpr int PW = 68;                 // pitch of the weights
  constexpr int NR = 1 + 2 * NP;         // row operands: dO, dv and V' in planes
  // in LDS dO has as many planes as the others (zeros), so that the tiles of dP
  // and dA are the same products
  constexpr int ROWS = 3 * NP * kB * PA;
  constexpr int TILES = 2 * NP * ST::BYTES, MAT = kB * PM;
  constexpr int S_BYTES = NP * MAT * SZ;  // dA + dA^T, in the place of the first tiles
  struct Weights { float w[2][kB][PW]; };
  struct Mats { T p[NP][MAT], pt[NP][MAT]; };
  union Rows { T rows[2][ROWS]; Weights wt; Mats m; __device__ Rows() {} };
  // Objects of their own: the compiler lets reads of one pair of tiles pass the
  // direct loads on their way into the other only where it knows them apart.
  __shared__ __attribute__((aligned(1024))) char tiles0[TILES > S_BYTES ? TILES : S_BYTES];
  __shared__ __attribute__((aligned(1024))) char tiles1[TILES];
  __shared__ __attribute__((aligned(16))) Rows sh;
  __shared__ double sg[kB];
  __shared__ float sx[NW][kB], sy[NW][kB], sw[NW][kB], sz[NW], sbeta[kB];
  T* const tag = nullptr;

  const int tid = threadIdx.x, lane = tid & 63, w = uniform_i(tid >> 6);
  const int b = blockIdx.x / p.blocks_max, blk = blockIdx.x % p.blocks_max, hk = blockIdx.y;
  int64_t tok0;
  int len, base;
  seq_span(p, b, tok0, len, base);
  if (blk * kB >= len) return;
  const int rows = min(kB, len - blk * kB);
  const int64_t row0 = tok0 + blk * kB;
  const int n = lane & 31, h2 = lane >> 5;
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;
  const int group = GROUPED ? p.heads / p.k_heads : 1;
  const int64_t key_slot = (int64_t)(base + blk) * p.k_heads + hk;

  f32x16 dq[2] = {zero16(), zero16()}, dk[2] = {zero16(), zero16()};
  for (int hh = 0; hh < group; ++hh) {
    const int h = hk * group + hh;
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    const T* SN = reinterpret_cast<const T*>(p.snap) + slot * (NP * D * D);
    const T* DN = reinterpret_cast<const T*>(p.dsnap) + slot * (NP * D * D);
    TileLoads<T, ST, NW> sloads;
    sloads.init(D, lane);
    constexpr int CHUNKS = kB * (DV / 8);  // of 8 elements in a row operand, a whole number of waves
    constexpr int RN = (NR * CHUNKS + 2 * D - 1) / (2 * D);
    const int cr = (tid % CHUNKS) / 2, cj = tid % 2 * 8;  // row and column of the thread's chunks
    Raw8<T> raw[RN];
    auto operand_of = [&](int i) { return uniform_i((tid + i * 2 * D) / CHUNKS); };
    auto ask = [&](int d0, char* tiles) {
#pragma unroll
      for (int pl = 0; pl < NP; ++pl) {
        sloads.issue(tiles + pl * ST::BYTES, SN + pl * D * D, D, d0, w);
        sloads.issue(tiles + (NP + pl) * ST::BYTES, DN + pl * D * D, D, d0, w);
      }
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int m = operand_of(i);
        const T* src = reinterpret_cast<const T*>(m == 0 ? p.dout : m == 1 ? p.dv : NP > 1 && m == 2 ? p.dv_rest : p.u);
        if (m > NP) src += (m - 1 - NP) * (int64_t)p.total * vs;
        const auto rs = scalar_rsrc(src + row0 * vs + h * D, m < NR ? rows * (uint32_t)vs * SZ : 0);
        raw[i] = __builtin_bit_cast(Raw8<T>, buf_frag(rs, (cr * (uint32_t)vs + cj) * SZ, d0 * SZ, tag));
      }
    };
    // columns within 16 in the order of the column fragments: 0-3, 8-11, 4-7, 12-15
    auto put_rows = [&](int buf) {
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int m = operand_of(i);
        if (m < NR) {
          const frag_t<T> x = __builtin_bit_cast(frag_t<T>, raw[i]);
          T* to = sh.rows[buf] + ((m ? NP + m - 1 : 0) * kB + cr) * PA + cj / 2;
          *reinterpret_cast<vec4_t<T>*>(to) = vec4_t<T>{x[0], x[1], x[2], x[3]};
          *reinterpret_cast<vec4_t<T>*>(to + 8) = vec4_t<T>{x[4], x[5], x[6], x[7]};
        }
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
    if constexpr (NP > 1) {
      for (int i = tid; i < 2 * kB * PA / 8; i += 2 * D)
        store8_zero(sh.rows[i / (kB * PA / 8)] + kB * PA + i % (kB * PA / 8) * 8);
    }

    f32x16 acc[TW];  // [s][r]: V' dO^T and V' dv^T
#pragma unroll
    for (int k = 0; k < TW; ++k) acc[k] = zero16();
    // dO S^T, V' dS^T and dv S^T over the value columns, and <S, dS>
    f32x16 a0[2] = {zero16(), zero16()}, a1[2] = {zero16(), zero16()}, a2[2] = {zero16(), zero16()};
    float z = 0.f;
    auto step = [&](int d0, const char* tiles, char* next, int buf) {
      put_rows(buf);
      __builtin_amdgcn_s_waitcnt(0);  // the tiles
      lds_barrier();
      if (d0 + DV < D) ask(d0 + DV, next);
      auto row = [&](int plane, int rt) {
        return lds_row8(sh.rows[buf] + (plane * kB + 32 * rt + n) * PA + 8 * h2);
      };
      frag_t<T> fs[NP], fd[NP];
#pragma unroll
      for (int pl = 0; pl < NP; ++pl) {
        fs[pl] = state_tile_col8<ST>(tiles + pl * ST::BYTES, 0, 32 * w, lane, tag);
        fd[pl] = state_tile_col8<ST>(tiles + (NP + pl) * ST::BYTES, 0, 32 * w, lane, tag);
      }
      // (products of two rests are below 2^-17 of the first and left out)
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const frag_t<T> x = row(0, rt);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const frag_t<T> dv = row(NP + i, rt), u = row(2 * NP + i, rt);
          a0[rt] = mma32(x, fs[i], a0[rt]);
#pragma unroll
          for (int j = 0; i + j < NP; ++j) {
            a2[rt] = mma32(dv, fs[j], a2[rt]);
            a1[rt] = mma32(u, fd[j], a1[rt]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < TW; ++k) {
        const int task = w + k * NW, which = task >> 2, rt = task >> 1 & 1, st = task & 1;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; i + j < NP; ++j)
            acc[k] = mma32(row(2 * NP + i, st), row(which * NP + j, rt), acc[k]);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; i + j < NP; ++j) z = dot_frag(fs[i], fd[j], z);
    };
    ask(0, tiles0);
    for (int d0 = 0; d0 < D; d0 += 2 * DV) {
      step(d0, tiles0, tiles1, 0);
      step(d0 + DV, tiles1, tiles0, 1);
    }
    frag_t<T> fq[4], fk[4];  // queries and keys by columns, the wave's 32
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int64_t at = key_slot * (kB * D) + 8 * lane + column_frag(w, ks);
      fq[ks] = *reinterpret_cast<const frag_t<T>*>(reinterpret_cast<const T*>(p.qc) + at);
      fk[ks] = *reinterpret_cast<const frag_t<T>*>(reinterpret_cast<const T*>(p.kc) + at);
    }
    __syncthreads();  // the stage has been read
    // dP and dA in place of the sums, and their weights
#pragma unroll
    for (int k = 0; k < TW; ++k) {
      const int task = w + k * NW, which = task >> 2, r = 32 * (task >> 1 & 1) + n, s0 = 32 * (task & 1) + 4 * h2;
      const float* pairs = p.pairs + (key_slot * 2 + which) * (kB * kB) + r * kB + s0;
      const double gr = sg[r];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 pair = *reinterpret_cast<const f32x4*>(pairs + 8 * q);
        f32x4 wt;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int s = s0 + 8 * q + i;
          const float e = __builtin_amdgcn_exp2f((float)((gr - sg[s]) * 1.4426950408889634));
          float x = acc[k][4 * q + i];
          if (which && s == r) sbeta[r] = x;
          x = which ? -e * x : p.scale * e * x;
          wt[i] = s < r ? pair[i] * x : 0.f;
          acc[k][4 * q + i] = s < r || (s == r && !which) ? x : 0.f;
        }
        *reinterpret_cast<f32x4*>(&sh.wt.w[which][r][s0 + 8 * q]) = wt;
      }
    }
    const float* vec = p.vec + slot * (4 * kB);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 32 * rt + 8 * q + 4 * h2;
        const f32x4 eg = *reinterpret_cast<const f32x4*>(vec + r), el = *reinterpret_cast<const f32x4*>(vec + kB + r);
        f32x4 xs, ys;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * q + i;
          const float x = p.scale * eg[i] * a0[rt][e], y = el[i] * a1[rt][e], v = eg[i] * a2[rt][e];
          const float key = (float)fk[2 * rt + e / 8][e % 8];
          xs[i] = (float)fq[2 * rt + e / 8][e % 8] * x - key * v;
          ys[i] = key * y;
          dq[rt][e] = GROUPED ? dq[rt][e] + x : x;
          dk[rt][e] = GROUPED ? dk[rt][e] + (y - v) : y - v;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xs[i] = sum_lanes<32>(xs[i]);
          ys[i] = sum_lanes<32>(ys[i]);
        }
        if (n == 0) {
          *reinterpret_cast<f32x4*>(&sx[w][r]) = xs;
          *reinterpret_cast<f32x4*>(&sy[w][r]) = ys;
        }
      }
    z = sum64(z);
    if (lane == 0) sz[w] = z;
    __syncthreads();
    // weights between tokens before t and tokens from t on, for t = lane
    {
      float sum = 0.f;
#pragma unroll 4
      for (int r = w; r < kB; r += NW) {
        const int s = lane > 0 ? lane - 1 : 0;
        const float x = scan64(lane > 0 ? sh.wt.w[0][r][s] + sh.wt.w[1][r][s] : 0.f, lane);
        sum += lane <= r ? x : 0.f;
      }
      sw[w][lane] = sum;
    }
    __syncthreads();
    if (w == 0) {
      float x = 0.f, y = 0.f, sum = 0.f, zs = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        x += sx[i][63 - lane];  // tokens from t on: summed from the last, in reversed lanes
        y += lane ? sy[i][lane - 1] : 0.f;
        sum += sw[i][lane];
        zs += sz[i];
      }
      x = __shfl(scan64(x, lane), 63 - lane, 64);
      const float through = vec[kB - 1];  // exp(G_last)
      sum += x + scan64(y, lane) + (through == 0.f ? 0.f : through * zs);
      if (lane < rows) {
        const int64_t at = (row0 + lane) * p.heads + h;
        // a factor of 0 in 32 bits: no term is left, but those that are not finite
        const bool none = (blk + lane == 0 && !p.state_in) || p.log_decay[at] < kZeroLogDecay;
        p.d_log_decay[at] = none ? 0.f : sum;
        const float beta = vec[2 * kB + lane];
        p.d_beta[at] = sbeta[lane] / beta / beta;
      }
    }
    // dP (both ways round) and dA + dA^T as operands, in planes
    T* smat = reinterpret_cast<T*>(tiles0);
#pragma unroll
    for (int k = 0; k < TW; ++k) {
      const int task = w + k * NW, which = task >> 2, rt = task >> 1 & 1, st = task & 1;
      const int r = 32 * rt + n, s0 = 32 * st + 4 * h2;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 x = {acc[k][4 * q], acc[k][4 * q + 1], acc[k][4 * q + 2], acc[k][4 * q + 3]};
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
          vec4_t<T> y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = (T)x[i];
            x[i] -= (float)y[i];
          }
          if (which == 0) {
            *reinterpret_cast<vec4_t<T>*>(&sh.m.p[pl][r * PM + s0 + 8 * q]) = y;
#pragma unroll
            for (int i = 0; i < 4; ++i) sh.m.pt[pl][(s0 + 8 * q + i) * PM + r] = y[i];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int s = s0 + 8 * q + i;
              if (s <= r) {
                smat[pl * MAT + r * PM + s] = y[i];
                smat[pl * MAT + s * PM + r] = y[i];
              }
            }
          }
        }
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
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
          dk[rt] = mma32(mrow(sh.m.pt[pl], rt, ks), fq[ks], dk[rt]);
          dq[rt] = mma32(mrow(sh.m.p[pl], rt, ks), fk[ks], dq[rt]);
          dk[rt] = mma32(mrow(smat + pl * MAT, rt, ks), fk[ks], dk[rt]);
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
