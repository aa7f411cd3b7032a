// Gated delta rule, one decode step for a batch of single tokens, the state in
// place:
//     S' = a S,  u = beta (v - S'^T k),  S <- S' + k u^T,  o = scale S^T q.
// Bound by the state's stream: D x D fp32 values read and written a head. A
// workgroup holds COLS value columns of a head (all D key rows) in registers,
// so that the state is read once: S'^T k and S'^T q are both summed on the way
// in, o = scale (S'^T q + (k . q) u) needs no second pass, and the new state
// leaves from the registers. 385 us for 256 sequences of 16 heads of 256 (2.1
// GB: 5.5 TB/s, where a large copy reaches 5.2); 5.2 us for one sequence (64
// workgroups), which is the latency of load, sum and store.
#include "common.hpp"
#include "delta.hpp"

namespace ret {

template <typename T, int D, int COLS, bool STREAM>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
  constexpr int CQ = COLS / 4;     // threads across a row (float4 each)
  constexpr int RG = 256 / CQ;     // row groups
  constexpr int RPT = D / RG;      // rows of a thread
  static_assert(RPT >= 1, "every thread has a row");
  constexpr int SLICES = D / COLS;
  __shared__ __attribute__((aligned(16))) float pk[RG][COLS], pq[RG][COLS], su[COLS];
  __shared__ float skq[RG];
  const int tid = threadIdx.x;
  const int slice = blockIdx.x % SLICES, bh = blockIdx.x / SLICES, h = bh % p.heads, b = bh / p.heads;
  const int hk = h / (p.heads / p.k_heads);
  int slot = b;
  T* o = reinterpret_cast<T*>(p.o) + (int64_t)bh * D + slice * COLS;
  if (p.slots) {
    // a slot outside the pool, or one that an earlier sequence of the batch has, is inactive
    slot = p.slots[b];
    bool taken = slot < 0 || slot >= p.num_slots;
    for (int i = tid; i < b; i += 256) taken |= p.slots[i] == slot;
    if (__syncthreads_or(taken)) {
      for (int i = tid; i < COLS; i += 256) o[i] = (T)0.f;
      return;
    }
  }
  const int cq = tid % CQ, rg = tid / CQ;
  float* S = p.state + ((int64_t)slot * p.heads + h) * D * D + (int64_t)rg * D + slice * COLS + 4 * cq;
  f32x4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const f32x4* at = reinterpret_cast<const f32x4*>(S + (int64_t)i * RG * D);
    s[i] = STREAM ? __builtin_nontemporal_load(at) : *at;
  }
  const int64_t qk = ((int64_t)b * p.k_heads + hk) * D;
  const T* q = reinterpret_cast<const T*>(p.q) + qk;
  const T* k = reinterpret_cast<const T*>(p.k) + qk;
  float kr[RPT], kq = 0.f;
  f32x4 ak = {0.f, 0.f, 0.f, 0.f}, aq = ak;
  float qr[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    kr[i] = (float)k[rg + i * RG];
    qr[i] = (float)q[rg + i * RG];
    kq += kr[i] * qr[i];
  }
  const float a = expf(p.log_decay[bh]), beta = p.beta[bh];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = a == 0.f ? 0.f : a * s[i][e];  // forgotten, NaN and infinity too
    ak += kr[i] * s[i];
    aq += qr[i] * s[i];
  }
  *reinterpret_cast<f32x4*>(&pk[rg][4 * cq]) = ak;
  *reinterpret_cast<f32x4*>(&pq[rg][4 * cq]) = aq;
  if (cq == 0) skq[rg] = kq;
  __syncthreads();
  if (tid < COLS) {
    float sk = 0.f, sq = 0.f, w = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      sk += pk[r][tid];
      sq += pq[r][tid];
      w += skq[r];
    }
    const float u = beta * ((float)reinterpret_cast<const T*>(p.v)[(int64_t)bh * D + slice * COLS + tid] - sk);
    su[tid] = u;
    o[tid] = (T)(p.scale * (sq + w * u));
  }
  __syncthreads();
  const f32x4 u = *reinterpret_cast<const f32x4*>(&su[4 * cq]);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    s[i] += kr[i] * u;
    f32x4* at = reinterpret_cast<f32x4*>(S + (int64_t)i * RG * D);
    if constexpr (STREAM)
      __builtin_nontemporal_store(s[i], at);
    else
      *at = s[i];
  }
}

// States above this size do not stay in the caches (256 MB behind the L2s) from
// one step to the next, and bypass them; smaller ones are found there again.
constexpr size_t kStreamBytes = size_t(512) << 20;

template <typename T, int D>
static hipError_t launch_step_t(const DeltaStepParams& p, hipStream_t stream) {
  constexpr int COLS = 64;
  const unsigned blocks = (unsigned)p.batch * p.heads * (D / COLS);
  if ((size_t)p.batch * p.heads * D * D * sizeof(float) > kStreamBytes)
    hipLaunchKernelGGL((delta_step_kernel<T, D, COLS, true>), dim3(blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((delta_step_kernel<T, D, COLS, false>), dim3(blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_delta_step(const DeltaStepParams& p, int d, int dtype, hipStream_t stream) {
  if (dtype == 1) {
    switch (d) {
      case 64: return launch_step_t<bf16, 64>(p, stream);
      case 128: return launch_step_t<bf16, 128>(p, stream);
      case 256: return launch_step_t<bf16, 256>(p, stream);
    }
  } else {
    switch (d) {
      case 64: return launch_step_t<float, 64>(p, stream);
      case 128: return launch_step_t<float, 128>(p, stream);
      case 256: return launch_step_t<float, 256>(p, stream);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace ret
