// Rows of a norm in registers: how they are divided over lanes, their sums,
// the norm and its gradient.
#pragma once

#include "common.hpp"
#include "norms.hpp"

namespace ret {

// LPR lanes hold a row, 8 NV elements each. VEC: 16-byte accesses, lane l the
// elements 8 (v LPR + l) .. + 7; else single elements, j LPR + l (widths that
// are no multiple of 8 leave rows unaligned). A workgroup of 256 lanes (or LPR)
// holds RPB rows.
template <typename T, int LPR_, int NV, bool VEC>
struct NormRow {
  static constexpr int LPR = LPR_, E = 8 * NV;
  static constexpr int THREADS = LPR > 256 ? LPR : 256;
  static constexpr int RPB = THREADS / LPR;

  template <typename U>
  __device__ static __forceinline__ void load(float* x, const U* row, int width, int l, bool keep = true) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = 8 * (v * LPR + l);
        F8 y = {};
        if (keep && at < width) y = load8(row + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * v + e] = y.x[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = keep && j * LPR + l < width ? (float)row[j * LPR + l] : 0.f;
    }
  }
  // the lane's part of a row as it lies in memory, so that a row can be on its
  // way while another is worked on
  struct Raw { Raw8<T> v[VEC ? NV : 1]; T e[VEC ? 1 : E]; };
  __device__ static __forceinline__ void ask(Raw& r, const T* row, int width, int l, bool keep) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = 8 * (v * LPR + l);
        r.v[v] = Raw8<T>{};
        if (keep && at < width) r.v[v] = ld_raw8(row + at);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) r.e[j] = keep && j * LPR + l < width ? row[j * LPR + l] : (T)0.f;
    }
  }
  __device__ static __forceinline__ void take(float* x, const Raw& r) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const F8 y = unpack8(r.v[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[8 * v + e] = y.x[e];
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = (float)r.e[j];
    }
  }
  template <typename U>
  __device__ static __forceinline__ void store(U* row, const float* x, int width, int l) {
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = 8 * (v * LPR + l);
        F8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.x[e] = x[8 * v + e];
        if (at < width) store8(row + at, y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j * LPR + l < width) row[j * LPR + l] = (U)x[j];
    }
  }
  // whether element j of the lane exists
  __device__ static __forceinline__ bool inside(int j, int width, int l) {
    return (VEC ? 8 * ((j / 8) * LPR + l) : j * LPR + l) < width;
  }
};

// Sums over a row's lanes, N at a time. Rows of more than a wave go through
// LDS with one barrier a sum: `turn` alternates between two halves of `sh`, so
// a half is written again only after everybody has passed the barrier that
// follows its reads. Every lane of the workgroup calls it.
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float* sh, int& turn) {
  if constexpr (LPR <= 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sum_lanes<LPR>(s[i]);
  } else {
    constexpr int WPR = LPR / 64;
    const int wave = threadIdx.x >> 6;
    float* at = sh + turn * 32;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = sum_lanes<64>(s[i]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) at[wave * N + i] = s[i];
    }
    lds_barrier();  // (rows on their way from memory stay so)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s[i] += at[(wave / WPR * WPR + w) * N + i];
    }
  }
}

// x becomes (x - mean) / deviation (mean 0 unless `center`); returns the
// inverse deviation. The variance is summed from the centred values.
template <typename R>
__device__ __forceinline__ float normalize(float* x, int width, int center, float eps, int l, float* sh, int& turn) {
  const float inv = 1.f / width;
  if (center) {
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < R::E; ++j) s[0] += x[j];
    row_sums<R::LPR>(s, sh, turn);
#pragma unroll
    for (int j = 0; j < R::E; ++j) x[j] = R::inside(j, width, l) ? x[j] - s[0] * inv : 0.f;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < R::E; ++j) s[0] += x[j] * x[j];
  row_sums<R::LPR>(s, sh, turn);
  const float rstd = rsqrtf(s[0] * inv + eps);
#pragma unroll
  for (int j = 0; j < R::E; ++j) x[j] *= rstd;
  return rstd;
}

// g, the gradient of the normalised row n, becomes the row's own.
template <typename R>
__device__ __forceinline__ void normalize_grad(float* g, const float* n, float rstd, int width, int center, float* sh,
                                               int& turn) {
  const float inv = 1.f / width;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < R::E; ++j) {
    s[0] += g[j] * n[j];
    s[1] += g[j];
  }
  row_sums<R::LPR>(s, sh, turn);
  const float a = s[0] * inv, b = center ? s[1] * inv : 0.f;
#pragma unroll
  for (int j = 0; j < R::E; ++j) g[j] = rstd * (g[j] - b - n[j] * a);
}

// f(NormRow of the width's division) for rows of `width` elements. The backward
// (BWD) holds a dozen rows' worth of registers, so its rows of 4097 to 8192 are
// spread over 512 lanes (256 registers each), not 1024 (128, of which 72 more
// spill). That does not hold them all either: the residual norm's backward spills
// 46 registers of a lane (bf16) or 109 (fp32) there, and above 8192, where a row
// takes the 1024 lanes a workgroup has, 304 or 423; the head norm's 217 or 168
// there. Measured with all weights: 5.3 and 4.2 TB/s (fp32, bf16) at 4096, 2.6 and
// 2.8 at 8192, 0.8 and 0.7 at 16384; the head norm's backward 5.2 and 4.6 at
// 8192, 2.1 and 1.6 at 16384. Widths that are no multiple of 8 take single
// elements: the residual norm's forward 4.5 and 1.4 TB/s at 16380, 5.2 and 4.6 at
// 16384.
template <typename T, bool BWD, typename F>
hipError_t with_rows(int width, bool vec, F&& f) {
#define RET_NORM_CASE(LIMIT, LPR, NV) \
  if (width <= LIMIT) return vec ? f(NormRow<T, LPR, NV, true>{}) : f(NormRow<T, LPR, NV, false>{});
  RET_NORM_CASE(64, 8, 1)
  RET_NORM_CASE(128, 16, 1)
  RET_NORM_CASE(256, 32, 1)
  RET_NORM_CASE(512, 64, 1)
  RET_NORM_CASE(1024, 128, 1)
  RET_NORM_CASE(2048, 256, 1)
  RET_NORM_CASE(4096, 512, 1)
  RET_NORM_CASE(8192, (BWD ? 512 : 1024), (BWD ? 2 : 1))
  RET_NORM_CASE(kMaxNormWidth, 1024, 2)
#undef RET_NORM_CASE
  return hipErrorInvalidValue;
}

}  // namespace ret
