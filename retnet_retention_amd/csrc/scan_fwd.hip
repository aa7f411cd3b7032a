// Gated linear recurrence, forward: per channel
//     h_t = a_t h_(t-1) + m_t sigmoid(gate_t) x_t,   a_t = exp(la_t),
// la_t given, or -rate sigmoid(decay_t); m_t = sqrt(1 - a_t^2) or 1.
// Bound by memory (8 bytes an element in bf16 with both gates) with the gates'
// arithmetic close behind. Every element is read once: a workgroup holds 256 tokens
// of 64 channels in registers, as factors a and inputs u, a wave two segments of 16
// tokens: side by side in its half waves where lanes take pairs of bf16 channels, one
// after the other with single channels (so that both give the same bits). Each
// segment folds its tokens to one factor A and one input U, these meet in LDS, and
// one wave, a lane a channel, runs them into states before each segment. The
// state before the tile comes from the tile before it, as a word in memory that this
// wave waits for; then every segment runs its tokens from its state and stores them.
// Waiting one after the other takes 0.65 us a tile, less than the tiles of a
// long sequence take at the memory's rate unless it is narrower than some 1000
// channels; so tiles are long, 256 tokens. Where factors' products are no normal numbers
// (256 tokens that forget a third of the state each) the wave that joins forms them again with
// exponents, beside the others' inputs: with rates up to 10 2 x 8192 x 4096 takes 120 us, not
// 115, 4 x 2048 x 2560 41, not 38.5; with rates up to 0.5 nothing.
// Measured in bf16 with both gates, kernel alone: 2 x 8192 x 4096 109 to 118 us (4.5 to 4.9 TB/s; a
// copy reaches 5.07), 4 x 2048 x 2560 with the states kept 43 us, 4 x 8192 x 4100 297 us (rows
// that end inside a line); calls of 1 x 16384 x 8192 197 us (5.4 TB/s), 1 x 32768 x 1024 88 us
// (the chain of 128 tiles), 1 x 131072 x 2560 542 us (5.0 TB/s); fp32, 2 x 8192 x 2048 111 us
// (4.8 TB/s). Bound by memory, with 34 vector instructions for 64 elements, 63 % of the SIMDs'
// cycles, close behind. Without any arithmetic or wait it took 120 us when it took 123, before
// neighbouring groups shared an XCD; segments of 8 tokens in 1024 threads, twice the waves,
// the same 123. Neither was measured again since.
#include <algorithm>

#include "scan_common.hpp"

// The variants of a kernel give the same bits: fused multiply-adds only where they are written.
#pragma clang fp contract(off)

namespace ret {

constexpr int kSegment = 16;  // tokens

// TILE: kScanTile, or kScanOnly where no sequence has more than that. Without the bound of
// 128 registers fp32 inputs with a gate and log decays take 144, and a CU one workgroup.
template <typename T, bool GATES, bool IGATE, bool NORM, int V, int TILE>
__global__ __launch_bounds__(TILE * 2, sizeof(T) == 4 && !GATES ? 4 : 2) void scan_fwd_kernel(ScanParams p) {
  using D = std::conditional_t<GATES, T, float>;
  constexpr int LW = kScanChannels / V, PARTS = 2 / V, L = kSegment * PARTS, SEGS = TILE / kSegment;
  // factors and inputs of the segments, and of what stands before each; exponents of products
  // that are no normal number; whether a wave has some
  constexpr int BEFORE = TILE == kScanOnly ? 1 : SEGS;
  __shared__ float s_a[SEGS][kScanChannels], s_u[SEGS][kScanChannels], s_h[kScanChannels];
  __shared__ float s_p[BEFORE][kScanChannels], s_pu[BEFORE][kScanChannels];
  __shared__ int s_e[SEGS][kScanChannels], s_pe[BEFORE][kScanChannels], s_odd[SEGS / 2];
  clear_errors(p);
  const Place at = place_of<false>(p, TILE);
  if (!at.any) return;
  int tok0, len;
  span_of(p, at.b, tok0, len);
  const int from = at.i * TILE;  // the tile's first token
  if (from >= len && !(at.i == 0 && len == 0)) return;
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int seg = wave * 2 + lane / LW, cl = lane % LW * V;  // the lane's first segment
  const int c0 = at.group * kScanChannels, c = min(c0 + cl, p.width - V);
  const bool inside = c0 + cl < p.width;
  const int left = len - from, n = left - seg * kSegment;  // tokens from the tile's, the lane's start on
  float a[L][V], u[L][V], A[PARTS][V], U[PARTS][V];

  auto fold = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int64_t row = (int64_t)tok0 + from;
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.x_stride;
    const D* decay = reinterpret_cast<const D*>(p.decay) + row * p.decay_stride;
    const T* gate = reinterpret_cast<const T*>(p.gate) + (IGATE ? row * p.gate_stride : 0);
    lane_raw<T, V> rx[L], rg[IGATE ? L : 1];
    lane_raw<D, V> rd[L];
    const int there = min(left, TILE);
    const Rows<T, V> xs(x, p.x_stride, there, p.width, seg * kSegment, c);
    const Rows<D, V> ds(decay, p.decay_stride, there, p.width, seg * kSegment, c);
    const Rows<T, V> gs(gate, p.gate_stride, there, p.width, seg * kSegment, c);
#pragma unroll
    for (int j = 0; j < L; ++j) {
      rx[j] = FULL ? xs.load(j) : xs.load_if(j);
      rd[j] = FULL ? ds.load(j) : ds.load_if(j);
      if constexpr (IGATE) rg[j] = FULL ? gs.load(j) : gs.load_if(j);
    }
    float rate[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      rate[e] = GATES ? p.rate[c + e] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float g[V];
      Lane<D, V>::get(rd[j], a[j]);
      Lane<T, V>::get(rx[j], u[j]);
      if constexpr (IGATE) Lane<T, V>::get(rg[j], g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float la = GATES ? -rate[e] * sigmoid_of(a[j][e], T()) : a[j][e];
        float rest;
        factor<T>(la, a[j][e], rest);
        if constexpr (IGATE) u[j][e] *= sigmoid_of(g[e], T());
        if constexpr (NORM) u[j][e] *= __builtin_amdgcn_sqrtf(rest);
        if (!FULL && j >= n) {  // behind the end
          a[j][e] = 1.f;
          u[j][e] = 0.f;
        }
        float &A1 = A[j / kSegment][e], &U1 = U[j / kSegment][e];
        U1 = fmaf(a[j][e], U1, u[j][e]);
        A1 *= a[j][e];
      }
    }
  };
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[k][e] = 1.f;
      U[k][e] = 0.f;
    }
  const bool full = left >= TILE;
  if (full)
    fold(std::true_type());
  else if (wave * 2 * kSegment < left)
    fold(std::false_type());
  // a product that is no normal number: exact, and inputs that forget what stood before them
  bool odd = false;
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) odd |= !is_normal(A[k][e]);
  odd = __any(odd);
  if (odd) {
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float& U1 = U[j / kSegment][e];
        U1 = j % kSegment ? step_or_forget(a[j][e], U1, u[j][e]) : u[j][e];
      }
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (!is_normal(A[k][e])) {
          Growing t;
          bool none = false;
#pragma unroll
          for (int j = 0; j < kSegment; ++j) {
            none |= a[k * kSegment + j][e] == 0.f;
            t.by(a[k * kSegment + j][e]);
          }
          A[k][e] = none ? 0.f : -t.m;
          s_e[seg + k][cl + e] = t.e;
        }
  }
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s_a[seg + k][cl + e] = A[k][e];
      s_u[seg + k][cl + e] = U[k][e];
    }
  if (lane == 0) s_odd[wave] = odd;
  __syncthreads();
  if (wave == 0) {
    const int ch = c0 + lane;
    const bool mine = ch < p.width, last = left <= TILE;
    const int64_t held = (int64_t)at.b * p.width + ch;
    const bool any_odd = __any(s_odd[lane % (SEGS / 2)]);
    float h = 0.f;
    if constexpr (TILE == kScanOnly) {
      // no state to wait for: the segments one after the other
      if (p.state_in && mine) h = p.state_in[held];
      auto walk = [&](auto some) {
#pragma unroll 8
        for (int s = 0; s < SEGS; ++s) {
          const float sa = s_a[s][lane], su = s_u[s][lane];
          s_u[s][lane] = h;
          h = decltype(some)::value ? step_over({sa, s_e[s][lane]}, h, su) : fmaf(sa, h, su);
        }
      };
      if (any_odd)
        walk(std::true_type());
      else
        walk(std::false_type());
      if (mine && p.state_out) p.state_out[held] = h;
    } else {
      float ta = 1.f, tu = 0.f, low = 1.f;
#pragma unroll
      for (int s = 0; s < SEGS; ++s) {
        const float sa = s_a[s][lane], su = s_u[s][lane];
        s_p[s][lane] = ta;
        s_pu[s][lane] = tu;
        tu = fmaf(sa, tu, su);
        ta *= sa;
        low = fminf(low, ta);
      }
      bool far = !is_normal(ta) || !is_normal(low);
      if (any_odd)
        for (int s = 0; s < SEGS; ++s) far |= !is_normal(s_a[s][lane]);
      const bool any_far = __any(far);
      Product total = {ta, 0};
      if (far) {
        Growing t;
        if (any_odd) {
          tu = 0.f;
#pragma unroll 4
          for (int s = 0; s < SEGS; ++s) {
            const Product one = {s_a[s][lane], s_e[s][lane]};
            s_p[s][lane] = -t.m;
            s_pe[s][lane] = t.e;
            s_pu[s][lane] = tu;
            tu = step_over(one, tu, s_u[s][lane]);
            t.by(one);
          }
        } else {  // (the inputs as they are: every segment's factor is a normal number)
#pragma unroll
          for (int s = 0; s < SEGS; ++s) {
            s_p[s][lane] = -t.m;
            s_pe[s][lane] = t.e;
            t.by(s_a[s][lane]);
          }
        }
        total = t.product();
      }
      if (at.i > 0)
        h = take_over(p.hand + (at.tile - 1) * p.width + ch, mine, p.ctrl);
      else if (p.state_in && mine)
        h = p.state_in[held];
      s_h[lane] = h;
      h = any_far ? step_over(total, h, tu) : fmaf(ta, h, tu);
      if (mine) {
        if (!last)
          hand_on(p.hand + at.tile * p.width + ch, h);
        else if (p.state_out)
          p.state_out[held] = h;
      }
    }
  }
  __syncthreads();
  if (!inside || n <= 0) return;
  float h0[PARTS][V];
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (TILE == kScanOnly) {
        h0[k][e] = s_u[seg + k][cl + e];
      } else {
        h0[k][e] = step_over(s_p[seg + k][cl + e], &s_pe[seg + k][cl + e], s_h[cl + e], s_pu[seg + k][cl + e]);
      }
    }
  if (p.kept && seg * kSegment % kScanBwdTile == 0) {
    float* kept = p.kept + (kept_row(p, at.b, tok0) + (from + seg * kSegment) / kScanBwdTile) * p.width + c;
#pragma unroll
    for (int e = 0; e < V; ++e) kept[e] = h0[0][e];
  }
  if (!p.o) return;
  const Rows<T, V> o(reinterpret_cast<T*>(p.o) + ((int64_t)tok0 + from) * p.width, p.width, min(left, TILE),
                     p.width, seg * kSegment, c);
  auto run = [&](auto full, auto forget) {
    float h[V];
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (j % kSegment == 0) h[e] = h0[j / kSegment][e];
        h[e] = decltype(forget)::value ? step_or_forget(a[j][e], h[e], u[j][e]) : fmaf(a[j][e], h[e], u[j][e]);
      }
      if (decltype(full)::value || j < n) o.store(j, h);
    }
  };
  if (odd)
    run(std::false_type(), std::true_type());
  else if (full)
    run(std::true_type(), std::false_type());
  else
    run(std::false_type(), std::false_type());
}

// Clears what the workgroups hand each other and checks packed bounds.
__global__ __launch_bounds__(256) void scan_prep_kernel(ScanParams p, int64_t words) {
  if (blockIdx.x == 0) {
    bool ok = true;
    if (p.cu)
      for (int i = threadIdx.x; i < p.batch; i += 256) {
        int t0, n;
        ok = clamp_span(p.cu[i], p.cu[i + 1], p.total, p.total, t0, n) && ok;
      }
    ok = __syncthreads_and(ok);
    for (int i = threadIdx.x; i < (p.hand ? (int)kScanCtrlBytes / 4 : 2); i += 256)
      if (i != 1) p.ctrl[i] = 0;
    if (threadIdx.x == 0 && !p.keep_error) p.ctrl[1] = ok ? 0 : 2;
  }
  const u32x4 zero = {0, 0, 0, 0};
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words / 2; i += (int64_t)gridDim.x * 256)
    reinterpret_cast<u32x4*>(p.hand)[i] = zero;
  if (words % 2 && blockIdx.x == 0 && threadIdx.x == 0) p.hand[words - 1] = 0;
}
hipError_t launch_scan_prep(const ScanParams& p, hipStream_t stream) {
  if (!p.hand && !p.cu) return hipSuccess;  // the kernels themselves clear the control word
  const int64_t words = p.hand ? (int64_t)p.tiles * p.width : 0, blocks = (words + 2047) / 2048;
  hipLaunchKernelGGL(scan_prep_kernel, dim3((unsigned)(blocks < 1 ? 1 : blocks > 1024 ? 1024 : blocks)), dim3(256), 0,
                     stream, p, words);
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void check_bounds_kernel(const int* cu, int batch, int total, int* ctrl) {
  bool ok = true;
  for (int i = threadIdx.x; i < batch; i += 256) {
    int t0, n;
    ok = clamp_span(cu[i], cu[i + 1], total, total, t0, n) && ok;
  }
  ok = __syncthreads_and(ok);
  if (threadIdx.x == 0) {
    ctrl[0] = 0;
    ctrl[1] = ok ? 0 : 2;
  }
}
hipError_t launch_check_bounds(const int* cu, int batch, int total, int* ctrl, hipStream_t stream) {
  hipLaunchKernelGGL(check_bounds_kernel, dim3(1), dim3(256), 0, stream, cu, batch, total, ctrl);
  return hipGetLastError();
}

template <typename T, bool GATES, bool IGATE, bool NORM, int V, int TILE>
static hipError_t launch_fwd(const ScanParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((scan_fwd_kernel<T, GATES, IGATE, NORM, V, TILE>), dim3(scan_grid(p)), dim3(TILE * 2), 0, stream,
                     p);
  return hipGetLastError();
}
template <typename T, int V, int TILE>
static hipError_t launch_fwd_v(const ScanParams& p, hipStream_t s) {
  const int which = (p.rate ? 4 : 0) + (p.gate ? 2 : 0) + (p.normalize ? 1 : 0);
  switch (which) {
    case 0: return launch_fwd<T, false, false, false, V, TILE>(p, s);
    case 1: return launch_fwd<T, false, false, true, V, TILE>(p, s);
    case 2: return launch_fwd<T, false, true, false, V, TILE>(p, s);
    case 3: return launch_fwd<T, false, true, true, V, TILE>(p, s);
    case 4: return launch_fwd<T, true, false, false, V, TILE>(p, s);
    case 5: return launch_fwd<T, true, false, true, V, TILE>(p, s);
    case 6: return launch_fwd<T, true, true, false, V, TILE>(p, s);
    default: return launch_fwd<T, true, true, true, V, TILE>(p, s);
  }
}
template <int TILE>
static hipError_t launch_fwd_t(const ScanParams& p, int dtype, hipStream_t stream) {
  const hipError_t e = launch_scan_prep(p, stream);
  if (e != hipSuccess) return e;
  if (dtype != 1) return launch_fwd_v<float, 1, TILE>(p, stream);
  return in_pairs(p) ? launch_fwd_v<bf16, 2, TILE>(p, stream) : launch_fwd_v<bf16, 1, TILE>(p, stream);
}
// A sequence of up to kScanOnly tokens as one tile spares the launch that clears the
// words, and a hop, but its workgroups fill a CU alone; taken where there is one for each
// CU at most. bf16, a whole call from a graph, as one and as two tiles: 1 x 257 x 1024 10.2
// and 10.8 us (from the host 13.3 and 16.4), 16 x 300 x 1024 12.4 and 15.0, 32 x 300 x
// 1024 24.9 and 23.2, 64 x 300 x 1024 44 and 41.
static bool in_one(const ScanParams& p) {
  const int groups = (p.width + kScanChannels - 1) / kScanChannels;
  // (its rows are addressed with 32 bits from its first one)
  const bool far = std::max({p.x_stride, p.decay_stride, p.gate_stride}) >= (int64_t)1 << 21;
  return p.hand && !far && !has_chain(p.seqlen, p.cu, p.total, kScanOnly) && (int64_t)p.batch * groups <= 256;
}
hipError_t launch_scan_fwd(const ScanParams& p, int dtype, hipStream_t stream) {
  if (!in_one(p)) return launch_fwd_t<kScanTile>(p, dtype, stream);
  ScanParams only = p;
  only.hand = nullptr;
  only.tiles = (int)tile_count(p.batch, p.seqlen, p.cu, p.total, kScanOnly);
  return launch_fwd_t<kScanOnly>(only, dtype, stream);
}

}  // namespace ret
