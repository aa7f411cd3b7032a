// Gated linear recurrence, forward: per channel
//     h_t = a_t h_(t-1) + m_t sigmoid(gate_t) x_t,   a_t = exp(la_t),
// la_t given, or -rate sigmoid(decay_t); m_t = sqrt(1 - a_t^2) or 1.
// A workgroup walks a sequence in tiles of 128 tokens for the 64 V channels of its
// lanes. Each wave holds 16 tokens of a tile in registers: it forms their factors
// and inputs, folds them to one factor A and one input U, and the waves' pairs meet
// in LDS; each then runs its tokens from the state that reaches it.
#include "scan_common.hpp"

namespace ret {

template <typename T, bool GATES, bool IGATE, bool NORM, int V, int L, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void scan_fwd_kernel(ScanParams p) {
  using D = std::conditional_t<GATES, T, float>;
  static_assert(L * WAVES == kScanTile, "");
  __shared__ float s_a[2][WAVES][64 * V], s_u[2][WAVES][64 * V];
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int groups = (p.width + 64 * V - 1) / (64 * V);
  const int b = blockIdx.x / groups, at = (blockIdx.x % groups * 64 + lane) * V;
  const bool inside = at < p.width;
  const int c = min(at, p.width - V);
  int tok0, len;
  span_of(p, b, tok0, len);
  float rate[V], carry[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    rate[e] = GATES ? p.rate[c + e] : 0.f;
    carry[e] = p.state_in ? p.state_in[(int64_t)b * p.width + c + e] : 0.f;
  }
  const int64_t first_tile = p.cu ? tok0 / kScanTile + b : (int64_t)b * ((p.seqlen + kScanTile - 1) / kScanTile);
  const T* x = reinterpret_cast<const T*>(p.x) + tok0 * p.x_stride;
  const D* decay = reinterpret_cast<const D*>(p.decay) + tok0 * p.decay_stride;
  const T* gate = reinterpret_cast<const T*>(p.gate) + (IGATE ? tok0 * p.gate_stride : 0);
  T* o = reinterpret_cast<T*>(p.o) + (int64_t)tok0 * p.width;
  int turn = 0;
  for (int base = 0; base < len; base += kScanTile, turn ^= 1) {
    if (p.kept && wave == 0 && inside) {
#pragma unroll
      for (int e = 0; e < V; ++e) p.kept[(first_tile + base / kScanTile) * p.width + c + e] = carry[e];
    }
    const int t0 = base + wave * L, n = min(max(len - t0, 0), L);
    lane_raw<T, V> rx[L], rg[IGATE ? L : 1];
    lane_raw<D, V> rd[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int t = min(t0 + j, len - 1);
      rx[j] = lane_load<T, V>(x + t * p.x_stride, c);
      rd[j] = lane_load<D, V>(decay + t * p.decay_stride, c);
      if constexpr (IGATE) rg[j] = lane_load<T, V>(gate + t * p.gate_stride, c);
    }
    float a[L][V], u[L][V], A[V], U[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = 1.f;
      U[e] = 0.f;
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
        float left;
        factor<T>(la, a[j][e], left);
        if constexpr (IGATE) u[j][e] *= sigmoid_of(g[e], T());
        if constexpr (NORM) u[j][e] *= __builtin_amdgcn_sqrtf(left);
        if (j >= n) {  // behind the end
          a[j][e] = 1.f;
          u[j][e] = 0.f;
        }
        U[e] = step_or_forget(a[j][e], U[e], u[j][e]);
        A[e] *= a[j][e];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s_a[turn][wave][lane * V + e] = A[e];
      s_u[turn][wave][lane * V + e] = U[e];
    }
    __syncthreads();
    float h[V];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (w == wave) h[e] = carry[e];
        carry[e] = step_or_forget(s_a[turn][w][lane * V + e], carry[e], s_u[turn][w][lane * V + e]);
      }
    }
    if (p.o) {
#pragma unroll
      for (int j = 0; j < L; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = step_or_forget(a[j][e], h[e], u[j][e]);
        if (j < n && inside) lane_store<T, V>(o + (int64_t)(t0 + j) * p.width, c, h);
      }
    }
  }
  if (p.state_out && wave == 0 && inside) {
#pragma unroll
    for (int e = 0; e < V; ++e) p.state_out[(int64_t)b * p.width + c + e] = carry[e];
  }
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

template <typename T, bool GATES, bool IGATE, bool NORM, int V>
static hipError_t launch_fwd(const ScanParams& p, hipStream_t stream) {
  constexpr int L = 16, WAVES = kScanTile / L;
  const int64_t groups = (p.width + 64 * V - 1) / (64 * V);
  hipLaunchKernelGGL((scan_fwd_kernel<T, GATES, IGATE, NORM, V, L, WAVES>), dim3((unsigned)(groups * p.batch)),
                     dim3(WAVES * 64), 0, stream, p);
  return hipGetLastError();
}
template <typename T, int V>
static hipError_t launch_fwd_v(const ScanParams& p, hipStream_t s) {
  const int which = (p.rate ? 4 : 0) + (p.gate ? 2 : 0) + (p.normalize ? 1 : 0);
  switch (which) {
    case 0: return launch_fwd<T, false, false, false, V>(p, s);
    case 1: return launch_fwd<T, false, false, true, V>(p, s);
    case 2: return launch_fwd<T, false, true, false, V>(p, s);
    case 3: return launch_fwd<T, false, true, true, V>(p, s);
    case 4: return launch_fwd<T, true, false, false, V>(p, s);
    case 5: return launch_fwd<T, true, false, true, V>(p, s);
    case 6: return launch_fwd<T, true, true, false, V>(p, s);
    default: return launch_fwd<T, true, true, true, V>(p, s);
  }
}
hipError_t launch_scan_fwd(const ScanParams& p, int dtype, hipStream_t stream) {
  if (p.cu) {
    const hipError_t e = launch_check_bounds(p.cu, p.batch, p.total, p.ctrl, stream);
    if (e != hipSuccess) return e;
  }
  if (dtype != 1) return launch_fwd_v<float, 1>(p, stream);
  return in_pairs(p) ? launch_fwd_v<bf16, 2>(p, stream) : launch_fwd_v<bf16, 1>(p, stream);
}

}  // namespace ret
