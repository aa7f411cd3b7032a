// Gradients of the gated delta rule's chunkwise form. The forward's walk is
// run again (delta_fwd.hip, which keeps V', the state at each block's start and
// the row sums o . dO); then, with dS+ the gradient of a block's final state,
//     dV' = e^(G_last - G) K dS+ + P^T dO,   dX = T^T dV',   dv = beta dX,
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
//     d beta_t = dX_t . V'_t / beta_t   (V' = beta times the prediction error).
#include "delta_common.hpp"

namespace ret {

hipError_t launch_delta_forward(const DeltaParams& p, int d, int dtype, bool grad, hipStream_t stream);

template <typename T, int D>
struct ReverseIn {
  using CS = ChainShape<T, D>;
  static constexpr int NP = Planes<T>::N;
  frag_t<T> k[2][4];                  // rows of K, the wave's 64 key columns
  frag_t<T> tt[NP][2], pt[NP][2];     // rows 16 w .. + 15 of T^T and P^T
  T v[CS::CG][4][2], dout[CS::CG][4][2], u[NP][CS::CG][4][2];
  f32x4 eg, el, beta;
  float last;
};

template <typename T, int D>
__device__ __forceinline__ void load_reverse(ReverseIn<T, D>& in, const DeltaParams& p, int64_t row0, int rows,
                                             int64_t slot, int h, int hk, int slice, int w, int lane) {
  using CS = ChainShape<T, D>;
  constexpr int NP = Planes<T>::N;
  const int n = lane & 31, h2 = lane >> 5, g16 = lane >> 4, c = lane & 15;
  const int64_t qs = (int64_t)p.k_heads * D, vs = (int64_t)p.heads * D;
  const float* vec = p.vec + slot * (4 * kB);
  const T* tm = reinterpret_cast<const T*>(p.tt) + slot * (NP * kB * kB) + (16 * w + c) * kB + 8 * g16;
  const T* pm = reinterpret_cast<const T*>(p.pt) + slot * (NP * kB * kB) + (16 * w + c) * kB + 8 * g16;
  if (w < CS::WAVES) {
    const T* K = reinterpret_cast<const T*>(p.k) + row0 * qs + hk * D + 64 * (w % CS::RG) + 8 * h2;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) in.k[rt][ks] = global_row8(K + (32 * rt + n) * qs + 16 * ks, 32 * rt + n < rows);
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (ks < (w >> 1)) continue;  // upper triangular
#pragma unroll
    for (int pl = 0; pl < NP; ++pl) {
      in.tt[pl][ks] = global_row8(tm + pl * kB * kB + 32 * ks, true);
      in.pt[pl][ks] = global_row8(pm + pl * kB * kB + 32 * ks, true);
    }
  }
  const int r4 = 16 * w + 4 * g16;
  const int64_t at = row0 * vs + h * D + slice * CS::SL + 2 * c, plane = (int64_t)p.total * vs;
  const T* V = reinterpret_cast<const T*>(p.v) + at;
  const T* DO = reinterpret_cast<const T*>(p.dout) + at;
  const T* U = reinterpret_cast<const T*>(p.u) + at;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int cg = 0; cg < CS::CG; ++cg)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t o = (r4 + i) * vs + 32 * cg + e;
        const bool keep = r4 + i < rows;
        in.v[cg][i][e] = keep ? V[o] : (T)0.f;
        in.dout[cg][i][e] = keep ? DO[o] : (T)0.f;
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) in.u[pl][cg][i][e] = keep ? U[pl * plane + o] : (T)0.f;
      }
  in.eg = *reinterpret_cast<const f32x4*>(vec + r4);
  in.el = *reinterpret_cast<const f32x4*>(vec + kB + r4);
  in.beta = *reinterpret_cast<const f32x4*>(vec + 2 * kB + r4);
  in.last = vec[kB - 1];
}

// The gradient of the state, from a sequence's last block to its first; the
// same division of work and the same three exchanges as delta_chain_kernel.
template <typename T, int D>
__global__ __launch_bounds__(256) void delta_reverse_kernel(DeltaParams p) {
  using CS = ChainShape<T, D>;
  using KT = typename CS::KTile;
  constexpr int NP = Planes<T>::N;
  T* const tag = nullptr;
  // fp32 at d = 256 has no room for a second tile: Q's products follow K's in the same one
  constexpr bool kTwoTiles = !(sizeof(T) == 4 && D == 256);
  __shared__ __attribute__((aligned(1024))) char kt[CS::WAVES * KT::BYTES], qt[kTwoTiles ? CS::WAVES * KT::BYTES : 16];
  __shared__ __attribute__((aligned(16))) f32x4 part_k[CS::WAVES * 512];
  __shared__ __attribute__((aligned(16))) T od[CS::OPLANE], oq[CS::OPND], ox[CS::OPND], ow[CS::OPND];

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
  const int krow = 64 * rg, vcol = slice * CS::SL + 32 * cg_w + n;
  f32x16 s[2] = {zero16(), zero16()};
  if (holds && p.d_state_out) {
    const float* si = p.d_state_out + (int64_t)bh * D * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = si[(krow + 32 * t + state_row(i, h2)) * D + vcol];
  }
  char* my_kt = kt + w * KT::BYTES;
  char* my_qt = kTwoTiles ? qt + w * KT::BYTES : my_kt;
  TileLoads<T, KT, 1> loads;
  loads.init(qs, lane);
  auto load_tile = [&](char* to, const void* from, int64_t row0, int rows) {
    const T* src = reinterpret_cast<const T*>(from) + row0 * qs + hk * D + krow;
    if (rows == kB)
      loads.issue(to, src, qs, 0, 0);
    else
      loads.issue_clamped(to, src, qs, 0, rows - 1, 0);
  };
  constexpr bool kAhead = sizeof(T) == 2;
  ReverseIn<T, D> in;
  if (kAhead && nblk) {
    const int last = nblk - 1;
    load_reverse<T, D>(in, p, tok0 + last * kB, len - last * kB, (int64_t)(base + last) * p.heads + h, h, hk, slice, w,
                       lane);
  }

  for (int blk = nblk - 1; blk >= 0; --blk) {
    const int64_t row0 = tok0 + (int64_t)blk * kB;
    const int rows = min(kB, len - blk * kB);
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    const int r4 = 16 * w + 4 * g16;
    if constexpr (!kAhead) load_reverse<T, D>(in, p, row0, rows, slot, h, hk, slice, w, lane);
    if (holds) {
      __builtin_amdgcn_s_waitcnt(kWaitLds);  // the last block's reads of the tiles
      load_tile(my_kt, p.k, row0, rows);
      if constexpr (kTwoTiles) load_tile(my_qt, p.q, row0, rows);
      const bool group_end = (blk + 1) % kDeltaGroup == 0 || blk == nblk - 1;
      if (group_end && (blk != nblk - 1 || p.d_state_out)) {
        // <state, its gradient> at the group's end, this wave's part
        const int64_t at = (((int64_t)(base / kDeltaGroup + b + blk / kDeltaGroup) * p.heads + h) * CS::NSL + slice) *
                               CS::WAVES + w;
        const float* an = p.anchor + at * 2048 + lane * 4;
        float dot = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(an + (4 * t + q) * 256);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += x[i] * s[t][4 * q + i];
          }
        dot = sum64(dot);
        if (lane == 0) p.adot[at] = dot;
      }
      f32x16 ksum[2] = {zero16(), zero16()};
#pragma unroll
      for (int t = 0; t < 2; ++t)
        static_for<2>([&](auto sl) {
          constexpr int SLI = decltype(sl)::value;
          const Split<T> f = split_acc<SLI>(s[t], tag);
          const int ks = 2 * t + SLI;
#pragma unroll
          for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) ksum[rt] = mma32(in.k[rt][ks], f.f[pl], ksum[rt]);
          T* sn = reinterpret_cast<T*>(p.dsnap) + (slot * D + vcol) * D + krow + 32 * t + 16 * SLI + 8 * h2;
          *reinterpret_cast<frag_t<T>*>(sn) = f.f[0];
        });
      put_partial(part_k, w, ksum, lane);
    }
    // dO of the quarter as the other waves' operand (exact in T)
#pragma unroll
    for (int ct = 0; ct < CS::CT; ++ct) {
      vec4_t<T> x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = in.dout[ct >> 1][i][ct & 1];
      *reinterpret_cast<vec4_t<T>*>(od + (16 * ct + c) * CS::PITCH + r4) = x;
    }
    __syncthreads();

    // dV' of the quarter
#pragma unroll
    for (int ct = 0; ct < CS::CT; ++ct) {
      f32x4 x = get_partial<CS::RG>(part_k, ct, 4 * w + g16, c);
      f32x4 xd;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = r4 + i < rows ? x[i] * in.el[i] : 0.f;
        xd[i] = p.scale * in.eg[i] * (float)in.dout[ct >> 1][i][ct & 1];
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < (w >> 1)) continue;
        const frag_t<T> df = lds_row8(od + (16 * ct + c) * CS::PITCH + 32 * ks + 8 * g16);
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) x = mma(in.pt[pl][ks], df, x);
      }
      put_opnd<CS::PITCH, CS::OPLANE>(ox, 16 * ct + c, r4, x);
      put_opnd<CS::PITCH, CS::OPLANE>(oq, 16 * ct + c, 16 * w + quad_place(g16), xd);
    }
    __syncthreads();

    // dX = T^T dV', dv = beta dX
    f32x4 vdv = zero4(), xu = zero4();
#pragma unroll
    for (int ct = 0; ct < CS::CT; ++ct) {
      f32x4 dx = zero4();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < (w >> 1)) continue;
        frag_t<T> tf[NP], xf[NP];
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
          tf[pl] = in.tt[pl][ks];
          xf[pl] = lds_row8(ox + pl * CS::OPLANE + (16 * ct + c) * CS::PITCH + 32 * ks + 8 * g16);
        }
        dx = mma_split2(tf, xf, dx, tag);
      }
      f32x4 ed;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float dv = in.beta[i] * dx[i];
        ed[i] = -in.eg[i] * dv;
        float u = 0.f;
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) u += (float)in.u[pl][ct >> 1][i][ct & 1];
        vdv[i] += dv * (float)in.v[ct >> 1][i][ct & 1];
        xu[i] += dx[i] * u;
        if (r4 + i < rows)
          reinterpret_cast<T*>(p.dv)[(row0 + r4 + i) * vs + h * D + slice * CS::SL + 32 * (ct >> 1) + 2 * c +
                                     (ct & 1)] = (T)dv;
      }
      put_opnd<CS::PITCH, CS::OPLANE>(ow, 16 * ct + c, 16 * w + quad_place(g16), ed);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vdv[i] = sum16(vdv[i]);
      xu[i] = sum16(xu[i]);
    }
    if (c == 0) {
      *reinterpret_cast<f32x4*>(p.vdv + (slot * CS::NSL + slice) * kB + r4) = vdv;
      *reinterpret_cast<f32x4*>(p.xu + (slot * CS::NSL + slice) * kB + r4) = xu;
    }
    const float last = in.last;
    __builtin_amdgcn_s_waitcnt(0);  // the tiles (LDS loads run past the compiler's counting)
    __syncthreads();

    ReverseIn<T, D> nx;
    if (kAhead && blk > 0)
      load_reverse<T, D>(nx, p, row0 - kB, kB, slot - p.heads, h, hk, slice, w, lane);
    if (holds) {
      auto add = [&](const char* tile, const T* opnd) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          frag_t<T> f[NP];
#pragma unroll
          for (int pl = 0; pl < NP; ++pl)
            f[pl] = lds_row8(opnd + pl * CS::OPLANE + (32 * cg_w + col_place(n)) * CS::PITCH + 16 * ks + 8 * h2);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const frag_t<T> a = state_col8<KT>(tile, 16 * ks, 32 * t, lane, tag);
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) s[t] = mma32(a, f[pl], s[t]);
          }
        }
      };
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] *= last;
      add(my_kt, ow);
      if constexpr (!kTwoTiles) {
        __builtin_amdgcn_s_waitcnt(kWaitLds);
        load_tile(my_qt, p.q, row0, rows);
        __builtin_amdgcn_s_waitcnt(0);
      }
      add(my_qt, oq);
    }
    if (kAhead && blk > 0) in = nx;
  }

  if (holds && p.d_state_in) {
    float* so = p.d_state_in + (int64_t)bh * D * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) so[(krow + 32 * t + state_row(i, h2)) * D + vcol] = s[t][i];
  }
}

// d q and d k of one block and key head, summed over the value heads that
// share it; wave w the key columns 32 w .. + 31.
template <typename T, int D>
__global__ __launch_bounds__(2 * D) void delta_qk_grad_kernel(DeltaParams p) {
  constexpr int NW = D / 32;
  constexpr int DV = 32;  // value rows of a state tile in LDS
  using ST = LTile<T, DV, D, kColTile>;
  using QT = LTile<T, kB, D, kColTile>;
  constexpr int PA = sizeof(T) == 2 ? 40 : 36;  // pitch of the row operands
  constexpr int PM = sizeof(T) == 2 ? 72 : 68;  // pitch of the 64 x 64 matrices
  constexpr int AROWS = 3 * kB * PA * (int)sizeof(T);
  constexpr int TILES = 2 * ST::BYTES + AROWS > QT::BYTES ? 2 * ST::BYTES + AROWS : QT::BYTES;
  __shared__ __attribute__((aligned(1024))) char buf[TILES];
  __shared__ __attribute__((aligned(16))) T mp[kB * PM], mpt[kB * PM], ms[kB * PM];
  __shared__ double sg[kB];
  T* const tag = nullptr;
  char* st_s = buf;
  char* st_d = buf + ST::BYTES;
  T* rows_a = reinterpret_cast<T*>(buf + 2 * ST::BYTES);  // [dO, dv, V'][64][PA]

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
  const int group = p.heads / p.k_heads;
  TileLoads<T, QT, NW> qloads;
  qloads.init(qs, lane);

  f32x16 dq[2] = {zero16(), zero16()}, dk[2] = {zero16(), zero16()};
  for (int hh = 0; hh < group; ++hh) {
    const int h = hk * group + hh;
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    const T* DO = reinterpret_cast<const T*>(p.dout) + row0 * vs + h * D;
    const T* DVp = reinterpret_cast<const T*>(p.dv) + row0 * vs + h * D;
    const T* U = reinterpret_cast<const T*>(p.u) + row0 * vs + h * D;
    __syncthreads();  // the last head's reads
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
    __syncthreads();
    // dP and dA: 8 tasks of 16 rows
    for (int task = w; task < 8; task += NW) {
      const int rb = task & 3, which = task >> 2;
      const T* A = (which ? DVp : DO) + (16 * rb + c) * vs + 8 * g16;
      const bool keep = 16 * rb + c < rows;
      f32x4 acc[4] = {zero4(), zero4(), zero4(), zero4()};
#pragma unroll 2
      for (int ks = 0; ks < D / 32; ++ks) {
        const frag_t<T> a = global_row8(A + 32 * ks, keep);
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
          if (ct > rb) break;
          const int r = 16 * ct + c;
          acc[ct] = mma(a, global_row8(U + r * vs + 8 * g16 + 32 * ks, r < rows), acc[ct]);
        }
      }
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        if (ct > rb) break;
        const int s = 16 * ct + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * rb + 4 * g16 + i;
          const float e = s <= r ? __builtin_amdgcn_exp2f((float)((sg[r] - sg[s]) * 1.4426950408889634)) : 0.f;
          if (which == 0 && s <= r) {
            const T x = (T)(p.scale * e * acc[ct][i]);
            mp[r * PM + s] = x;
            mpt[s * PM + r] = x;
          }
          if (which == 1 && s < r) {
            const T x = (T)(-e * acc[ct][i]);
            ms[r * PM + s] = x;
            ms[s * PM + r] = x;
          }
        }
      }
    }
    // dO S^T, V' dS^T and dv S^T over the value rows
    f32x16 a0[2] = {zero16(), zero16()}, a1[2] = {zero16(), zero16()}, a2[2] = {zero16(), zero16()};
    const T* SN = reinterpret_cast<const T*>(p.snap) + slot * D * D;
    const T* DN = reinterpret_cast<const T*>(p.dsnap) + slot * D * D;
    TileLoads<T, ST, NW> sloads;
    sloads.init(D, lane);
    for (int d0 = 0; d0 < D; d0 += DV) {
      __syncthreads();
      sloads.issue(st_s, SN, D, d0, w);
      sloads.issue(st_d, DN, D, d0, w);
      for (int i = tid; i < 3 * kB * (DV / 8); i += 2 * D) {
        const int m = i / (kB * (DV / 8)), r = i / (DV / 8) % kB, j = i % (DV / 8) * 8;
        const T* src = (m == 0 ? DO : m == 1 ? DVp : U) + r * vs + d0 + j;
        const frag_t<T> x = global_row8(src, r < rows);
        *reinterpret_cast<frag_t<T>*>(rows_a + (m * kB + r) * PA + j) = x;
      }
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < DV / 16; ++ks) {
        const frag_t<T> fs = tile_col8w<ST>(st_s, 16 * ks, 32 * w, lane, tag);
        const frag_t<T> fd = tile_col8w<ST>(st_d, 16 * ks, 32 * w, lane, tag);
        // the column fragments' order of the contraction
        auto row = [&](int m, int rt) {
          const T* at = rows_a + (m * kB + 32 * rt + n) * PA + 16 * ks + 4 * h2;
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
          dq[rt][4 * q + i] += p.scale * eg[i] * a0[rt][4 * q + i];
          dk[rt][4 * q + i] += el[i] * a1[rt][4 * q + i] - eg[i] * a2[rt][4 * q + i];
        }
      }
    // dP^T Q, then dP K and (dA + dA^T) K
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
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
      const T* src = reinterpret_cast<const T*>(pass ? p.k : p.q) + row0 * qs + hk * D;
      if (rows == kB)
        qloads.issue(buf, src, qs, 0, w);
      else
        qloads.issue_clamped(buf, src, qs, 0, rows - 1, w);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const frag_t<T> f = tile_col8w<QT>(buf, 16 * ks, 32 * w, lane, tag);
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          if (pass == 0) {
            dk[rt] = mma32(mrow(mpt, rt, ks), f, dk[rt]);
          } else {
            dq[rt] = mma32(mrow(mp, rt, ks), f, dq[rt]);
            dk[rt] = mma32(mrow(ms, rt, ks), f, dk[rt]);
          }
        }
      }
    }
  }
  T* DQ = reinterpret_cast<T*>(p.dq) + row0 * qs + hk * D + 32 * w + n;
  T* DK = reinterpret_cast<T*>(p.dk) + row0 * qs + hk * D + 32 * w + n;
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

// d log decay and d beta from the row sums, one wave per (group of blocks, head).
__global__ __launch_bounds__(64) void delta_gate_grad_kernel(DeltaParams p, int slices, int waves) {
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
    const float* ad = p.adot + ((int64_t)(base / kDeltaGroup + b + grp) * p.heads + h) * slices * waves;
    for (int i = 0; i < slices * waves; ++i) carry += ad[i];
  }
  for (int blk = last; blk >= grp * kDeltaGroup; --blk) {
    const int64_t slot = (int64_t)(base + blk) * p.heads + h;
    float d = 0.f, x = 0.f;
    for (int s = 0; s < slices; ++s) {
      const int64_t at = (slot * slices + s) * kB + lane;
      d += p.odo[at] - p.vdv[at];
      x += p.xu[at];
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
      // with no state before it the first token's decay acts on nothing: the
      // sum over the whole sequence is zero but for its rounding
      p.d_log_decay[at] = r == 0 && !p.state_in ? 0.f : d;
      p.d_beta[at] = x / p.vec[slot * (4 * kB) + 2 * kB + lane];
    }
  }
}

template <typename T, int D>
static hipError_t launch_backward(const DeltaParams& p, hipStream_t stream) {
  using CS = ChainShape<T, D>;
  hipLaunchKernelGGL((delta_reverse_kernel<T, D>), dim3(CS::NSL * p.batch * p.heads), dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_qk_grad_kernel<T, D>), dim3(p.batch * p.blocks_max, p.k_heads), dim3(2 * D), 0, stream, p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int groups = (p.blocks_max + kDeltaGroup - 1) / kDeltaGroup;
  hipLaunchKernelGGL(delta_gate_grad_kernel, dim3(p.batch * groups, p.heads), dim3(64), 0, stream, p, CS::NSL,
                     CS::WAVES);
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
