// Gated linear recurrence and short convolution, one decode step for a batch of
// single tokens, the state in place. Every element is on its own: the kernels are
// a launch and one trip to memory and back. Measured in bf16, kernels alone: 64 x 4096
// of the recurrence 3.4 us, 64 x 12288 of the convolution (4 taps) 4.0 us; a call from
// the host takes 9 to 10 us.
#include "scan_common.hpp"

namespace ret {

// Slot of sequence b, or -1: outside the pool, or an earlier sequence has it.
__device__ __forceinline__ int slot_of(const int* slots, int b, int num_slots) {
  if (!slots) return b;
  const int slot = slots[b];
  bool taken = slot < 0 || slot >= num_slots;
  for (int i = threadIdx.x; i < b; i += blockDim.x) taken |= slots[i] == slot;
  return __syncthreads_or(taken) ? -1 : slot;
}

template <typename T, bool GATES, int V>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepParams p) {
  using D = std::conditional_t<GATES, T, float>;
  const int b = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * V;
  const int slot = slot_of(p.slots, b, p.num_slots);
  if (c >= p.width) return;
  T* o = reinterpret_cast<T*>(p.o) + (int64_t)b * p.width;
  float h[V] = {};
  if (slot >= 0) {
    float* state = p.state + (int64_t)slot * p.width;
    float x[V], d[V], g[V];
    const auto rx = lane_load<T, V>(reinterpret_cast<const T*>(p.x) + b * p.x_stride, c);
    const auto rd = lane_load<D, V>(reinterpret_cast<const D*>(p.decay) + b * p.decay_stride, c);
    const auto rs = lane_load<float, V>(state, c);
    if (p.gate) Lane<T, V>::get(lane_load<T, V>(reinterpret_cast<const T*>(p.gate) + b * p.gate_stride, c), g);
    Lane<T, V>::get(rx, x);
    Lane<D, V>::get(rd, d);
    Lane<float, V>::get(rs, h);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a, left;
      factor<T>(GATES ? -p.rate[c + e] * sigmoid_of(d[e], T()) : d[e], a, left);
      float u = x[e];
      if (p.gate) u *= sigmoid_of(g[e], T());
      if (p.normalize) u *= __builtin_amdgcn_sqrtf(left);
      h[e] = step_or_forget(a, h[e], u);
    }
    lane_store<float, V>(state, c, h);
  }
  lane_store<T, V>(o, c, h);
}

template <typename T, int V>
static hipError_t launch_step(const ScanStepParams& p, hipStream_t stream) {
  const dim3 grid((p.width + 256 * V - 1) / (256 * V), p.batch);
  if (p.rate)
    hipLaunchKernelGGL((scan_step_kernel<T, true, V>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((scan_step_kernel<T, false, V>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}
hipError_t launch_scan_step(const ScanStepParams& p, int dtype, hipStream_t stream) {
  if (dtype != 1) return launch_step<float, 1>(p, stream);
  return in_pairs(p) ? launch_step<bf16, 2>(p, stream) : launch_step<bf16, 1>(p, stream);
}

template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepParams p) {
  const int b = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * V;
  const int slot = slot_of(p.slots, b, p.num_slots);
  if (c >= p.width) return;
  T* o = reinterpret_cast<T*>(p.o) + (int64_t)b * p.width;
  float z[V] = {};
  if (slot >= 0) {
    T* state = reinterpret_cast<T*>(p.state) + (int64_t)slot * (K - 1) * p.width;
    lane_raw<T, V> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j] = lane_load<T, V>(state + (int64_t)j * p.width, c);
    r[K - 1] = lane_load<T, V>(reinterpret_cast<const T*>(p.x) + b * p.x_stride, c);
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = p.bias ? p.bias[c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float x[V];
      Lane<T, V>::get(r[j], x);
#pragma unroll
      for (int e = 0; e < V; ++e) z[e] = fmaf(p.weight[(int64_t)(c + e) * K + j], x[e], z[e]);
    }
    if (p.swish) {
#pragma unroll
      for (int e = 0; e < V; ++e) z[e] *= sigmoid_of(z[e], T());
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      *reinterpret_cast<lane_raw<T, V>*>(state + (int64_t)j * p.width + c) = r[j + 1];
  }
  lane_store<T, V>(o, c, z);
}

template <typename T, int K>
static hipError_t launch_conv_step_k(const ConvStepParams& p, hipStream_t stream) {
  constexpr int V = sizeof(T) == 2 ? 2 : 1;
  if (V == 2 && !(p.width % 2 == 0 && pairs_aligned(p.x, p.x_stride, 2))) {
    hipLaunchKernelGGL((conv_step_kernel<T, K, 1>), dim3((p.width + 255) / 256, p.batch), dim3(256), 0, stream, p);
  } else {
    const dim3 grid((p.width + 256 * V - 1) / (256 * V), p.batch);
    hipLaunchKernelGGL((conv_step_kernel<T, K, V>), grid, dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}
template <typename T>
static hipError_t launch_conv_step_t(const ConvStepParams& p, int taps, hipStream_t stream) {
  switch (taps) {
    case 2: return launch_conv_step_k<T, 2>(p, stream);
    case 3: return launch_conv_step_k<T, 3>(p, stream);
    case 4: return launch_conv_step_k<T, 4>(p, stream);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_conv_step(const ConvStepParams& p, int taps, int dtype, hipStream_t stream) {
  return dtype == 1 ? launch_conv_step_t<bf16>(p, taps, stream) : launch_conv_step_t<float>(p, taps, stream);
}

}  // namespace ret
