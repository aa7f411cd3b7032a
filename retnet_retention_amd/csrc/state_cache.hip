// States of parked sessions in 8 bits. Blocks of 64 values of a state share a scale
//     scale = max |x| (1 / 127),   code = x / scale rounded to the nearest, halves to even,
// and are read back as code scale. Integers with a scale of their own every 64 values
// keep a state to half a 127th of its block's largest value; e4m3 of the same size
// keeps each value to a 16th of itself, five times worse over values of one
// size. Bound by memory: 4 bytes a value on one side, 1.06 on the other. Measured, 64
// states of 4 MiB, kernels alone: written in 83 us (4.1 TB/s), read back in 49
// (6.9 TB/s by the bytes: the codes just written come from the caches), read from 24 others' in 45.
#include "common.hpp"
#include "state_cache.hpp"

namespace ret {

// Slot `i` of a list, or -1 where it lies outside `n`.
__device__ __forceinline__ int64_t listed(const int* list, int i, int64_t n) {
  const int64_t s = list ? list[i] : i;
  return s < 0 || s >= n ? -1 : s;
}

// Whether an earlier sequence of the batch names the same slot of `list` and, with
// `source`, one of its `n` slots there.
__device__ __forceinline__ bool named_before(const int* list, int b, const int* source, int64_t n) {
  bool hit = false;
  if (list)
    for (int i = threadIdx.x; i < b; i += blockDim.x)
      hit |= list[i] == list[b] && (!source || (source[i] >= 0 && source[i] < n));
  return __syncthreads_or(hit);
}

// x / scale to the nearest integer, halves to even: the product with the reciprocal
// can round to the wrong side of a half, which the remainder (exact) tells.
__device__ __forceinline__ int code_of(float x, float scale, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, scale, x), half = 0.5f * scale;
  const bool odd = ((int)q & 1) != 0;
  if (r > half || (r == half && odd)) q += 1.f;
  if (r < -half || (r == -half && odd)) q -= 1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// 16 lanes take a block of 64 values, 4 values each; a workgroup 16 blocks at a time, 4
// times where it writes the cache, twice where it reads it, all of them on their way from
// memory together. 64 states of 4 MiB written with 2 / 4 / 8: 81 / 78 / 80 us; read
// with 1 / 2 / 4 / 8: 59 / 45 / 48 / 52 us.
constexpr int kWriteAtOnce = 4, kReadAtOnce = 2;
// `whole`: the states' rows are aligned to 4 values, so 4 are there or none
// STREAM: states past the caches
template <bool STREAM>
__device__ __forceinline__ f32x4 four_of(const float* x, int64_t v, int64_t values, bool whole) {
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  if (whole) {
    const f32x4* at = reinterpret_cast<const f32x4*>(x + v);
    if (v < values) y = STREAM ? __builtin_nontemporal_load(at) : *at;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v + e < values) y[e] = x[v + e];
  }
  return y;
}

template <bool STREAM>
__global__ __launch_bounds__(256) void state_cache_write_kernel(StateCacheParams p) {
  const int b = blockIdx.y;
  const int64_t to = listed(p.at, b, p.cache_slots), from = listed(p.slots, b, p.num_slots);
  if (to < 0 || from < 0) return;
  if (named_before(p.at, b, p.slots, p.num_slots)) return;
  const int64_t first = (int64_t)blockIdx.x * 16 * kWriteAtOnce + (threadIdx.x >> 4);
  const int64_t v0 = first * kCacheBlock + 4 * (threadIdx.x & 15);
  const float* x = p.state + from * p.values;
  int8_t* codes = p.codes + to * p.values;
  const bool whole = p.values % 4 == 0;
  f32x4 y[kWriteAtOnce];
#pragma unroll
  for (int k = 0; k < kWriteAtOnce; ++k) y[k] = four_of<STREAM>(x, v0 + k * 16 * kCacheBlock, p.values, whole);
#pragma unroll
  for (int k = 0; k < kWriteAtOnce; ++k) {
    const int64_t v = v0 + k * 16 * kCacheBlock, block = first + k * 16;
    // the largest magnitude by its bits: a NaN is above infinity
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(y[k][e]) & 0x7fffffffu);
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s, 64));
    // NaN or infinity: the block reads back as NaN
    const float scale =
        top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) * (1.f / 127.f);
    // a quotient's reciprocal stays finite if both sides of a tiny one are brought up (exact)
    const float up = scale < 0x1p-64f ? 0x1p+64f : 1.f, s = scale * up, inv = 1.f / s;
    uint32_t word = 0;
    if (scale > 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) word |= (uint32_t)(code_of(y[k][e] * up, s, inv) & 0xff) << (8 * e);
    }
    if (whole) {
      if (v < p.values) *reinterpret_cast<uint32_t*>(codes + v) = word;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + e < p.values) codes[v + e] = (int8_t)(word >> (8 * e));
    }
    if ((threadIdx.x & 15) == 0 && block < p.blocks) p.scales[to * p.blocks + block] = scale;
  }
}

template <bool STREAM>
__global__ __launch_bounds__(256) void state_cache_read_kernel(StateCacheParams p) {
  const int b = blockIdx.y;
  const int64_t from = listed(p.at, b, p.cache_slots), to = listed(p.slots, b, p.num_slots);
  if (to < 0) return;
  if (named_before(p.slots, b, nullptr, 0)) return;
  const int64_t first = (int64_t)blockIdx.x * 16 * kReadAtOnce + (threadIdx.x >> 4);
  const int64_t v0 = first * kCacheBlock + 4 * (threadIdx.x & 15);
  float* x = p.state + to * p.values;
  const bool whole = p.values % 4 == 0;
  float scale[kReadAtOnce] = {};
  uint32_t word[kReadAtOnce] = {};
  if (from >= 0) {
    const int8_t* codes = p.codes + from * p.values;
#pragma unroll
    for (int k = 0; k < kReadAtOnce; ++k) {
      const int64_t v = v0 + k * 16 * kCacheBlock, block = first + k * 16;
      if (block < p.blocks) scale[k] = p.scales[from * p.blocks + block];
      if (whole) {
        if (v < p.values) word[k] = *reinterpret_cast<const uint32_t*>(codes + v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v + e < p.values) word[k] |= (uint32_t)(uint8_t)codes[v + e] << (8 * e);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kReadAtOnce; ++k) {
    const int64_t v = v0 + k * 16 * kCacheBlock;
    f32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)(int8_t)(word[k] >> (8 * e)) * scale[k];
    if (whole) {
      f32x4* at = reinterpret_cast<f32x4*>(x + v);
      if (v < p.values) {
        if constexpr (STREAM)
          __builtin_nontemporal_store(y, at);
        else
          *at = y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + e < p.values) x[v + e] = y[e];
    }
  }
}

static dim3 grid_of(const StateCacheParams& p, int at_once) {
  return dim3((unsigned)((p.blocks + 16 * at_once - 1) / (16 * at_once)), (unsigned)p.batch);
}
// States that do not fit the cache behind the L2s (256 MB) cannot be found there
// by whoever reads them next, so they bypass it; smaller ones stay. Through it and past it,
// n states of 4 MiB, calls in us: written right after the decode step that made them, n = 32 /
// 48 / 56 / 64 / 80 / 128 38 / 51 / 60 / 72 / 103 / 166 and 39 / 52 / 58 / 65 / 82 / 139; read
// back from memory with a decode step after it 77 / 109 / 130 / 153 / 199 / 331 and 83 / 118 /
// 134 / 152 / 188 / 305.
constexpr size_t kStreamBytes = size_t(256) << 20;
static bool streams(const StateCacheParams& p) { return (size_t)p.batch * p.values * sizeof(float) >= kStreamBytes; }

hipError_t launch_state_cache_write(const StateCacheParams& p, hipStream_t stream) {
  if (streams(p))
    hipLaunchKernelGGL((state_cache_write_kernel<true>), grid_of(p, kWriteAtOnce), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((state_cache_write_kernel<false>), grid_of(p, kWriteAtOnce), dim3(256), 0, stream, p);
  return hipGetLastError();
}
hipError_t launch_state_cache_read(const StateCacheParams& p, hipStream_t stream) {
  if (streams(p))
    hipLaunchKernelGGL((state_cache_read_kernel<true>), grid_of(p, kReadAtOnce), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((state_cache_read_kernel<false>), grid_of(p, kReadAtOnce), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace ret
