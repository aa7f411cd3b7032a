// What the kernels of the gated recurrence and the short convolution share: the
// channels of a lane, packed sequences, and the recurrence's gates.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "scan.hpp"

#pragma clang fp contract(off)

namespace ret {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// V neighbouring channels of a token, as they lie in memory and as floats.
template <typename T, int V> struct Lane;
template <> struct Lane<bf16, 1> {
  using Raw = bf16;
  __device__ static __forceinline__ void get(Raw r, float* x) { x[0] = (float)r; }
  __device__ static __forceinline__ Raw put(const float* x) { return (bf16)x[0]; }
};
template <> struct Lane<bf16, 2> {
  using Raw = uint32_t;
  __device__ static __forceinline__ void get(Raw r, float* x) {
    x[0] = __uint_as_float(r << 16);
    x[1] = __uint_as_float(r & 0xffff0000u);
  }
  __device__ static __forceinline__ Raw put(const float* x) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(bf16)x[0], (bf16)x[1]});
  }
};
template <> struct Lane<float, 1> {
  using Raw = float;
  __device__ static __forceinline__ void get(Raw r, float* x) { x[0] = r; }
  __device__ static __forceinline__ Raw put(const float* x) { return x[0]; }
};
template <> struct Lane<float, 2> {
  typedef float Raw __attribute__((ext_vector_type(2)));
  __device__ static __forceinline__ void get(Raw r, float* x) {
    x[0] = r[0];
    x[1] = r[1];
  }
  __device__ static __forceinline__ Raw put(const float* x) { return Raw{x[0], x[1]}; }
};
template <typename T, int V>
using lane_raw = typename Lane<T, V>::Raw;

// `row`: a wave-uniform pointer; `at`: a lane's elements behind it, below 2^32 bytes
template <typename T, int V>
__device__ __forceinline__ lane_raw<T, V> lane_load(const T* row, uint32_t at) {
  return *reinterpret_cast<const lane_raw<T, V>*>(reinterpret_cast<const char*>(row) + at * (uint32_t)sizeof(T));
}
template <typename T, int V>
__device__ __forceinline__ void lane_store(T* row, uint32_t at, const float* x) {
  *reinterpret_cast<lane_raw<T, V>*>(reinterpret_cast<char*>(row) + at * (uint32_t)sizeof(T)) = Lane<T, V>::put(x);
}

// Rows of a tile behind a scalar descriptor of `rows` rows: a lane's offset stays, the
// row is a scalar offset, so that an access costs no address arithmetic. All below 2^32
// bytes (strides below 2^22 where a sequence has more than one token).
constexpr int kStreamed = 2;  // store policy: not kept in the caches
template <typename T, int V>
struct Rows {
  using Raw = lane_raw<T, V>;
  __amdgpu_buffer_rsrc_t rs;
  uint32_t at, step;  // bytes: the lane's, from a row to the next
  // `row`: the lane's first row behind `base`, `c` its channel; a lane that is not inside
  // is sent behind the end of dense rows (below 2^31 bytes), where a store is dropped
  __device__ __forceinline__ Rows(const T* base, int64_t stride, int rows, int width, int row, int c,
                                  bool inside = true)
      : rs(scalar_rsrc(base, (uint32_t)((rows - 1) * stride + width) * (uint32_t)sizeof(T))),
        at(inside ? (uint32_t)(row * (uint32_t)stride + c) * (uint32_t)sizeof(T) : 0x80000000u),
        step((uint32_t)stride * (uint32_t)sizeof(T)) {}
  // a row that is there; one that may be behind the end (then zeros)
  __device__ __forceinline__ Raw load(int j) const { return get(at, j * step); }
  __device__ __forceinline__ Raw load_if(int j) const { return get(at + j * step, 0); }
  template <int POLICY = 0>
  __device__ __forceinline__ void store(int j, const float* x) const {
    const Raw r = Lane<T, V>::put(x);
    if constexpr (sizeof(Raw) == 2)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, r), rs, at, j * step, POLICY);
    else if constexpr (sizeof(Raw) == 4)
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, r), rs, at, j * step, POLICY);
    else
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, r), rs, at, j * step, POLICY);
  }

 private:
  __device__ __forceinline__ Raw get(uint32_t lane, uint32_t scalar) const {
    if constexpr (sizeof(Raw) == 2)
      return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b16(rs, lane, scalar, 0));
    else if constexpr (sizeof(Raw) == 4)
      return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b32(rs, lane, scalar, 0));
    else
      return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b64(rs, lane, scalar, 0));
  }
};

// Whether a lane may take two bf16 channels of every tensor at once.
template <typename P>
inline bool in_pairs(const P& p) {
  return p.width % 2 == 0 && pairs_aligned(p.x, p.x_stride, 2) &&
         pairs_aligned(p.decay, p.decay_stride, p.rate ? 2 : 4) && pairs_aligned(p.gate, p.gate_stride, 2);
}

// First row and length of sequence b, inside the tensor for any bounds.
template <typename P>
__device__ __forceinline__ void span_of(const P& p, int b, int& tok0, int& len) {
  if (p.cu) {
    packed_span(p.cu, b, p.total, p.total, tok0, len);
  } else {
    tok0 = b * p.seqlen;
    len = p.seqlen;
  }
}

// Row of the kept states: before token 0 of sequence b.
template <typename P>
__device__ __forceinline__ int64_t kept_row(const P& p, int b, int tok0) {
  return p.cu ? tok0 / kScanBwdTile + b : (int64_t)b * ((p.seqlen + kScanBwdTile - 1) / kScanBwdTile);
}

// Tile `j` as sequence b and its tile i, for tiles numbered as scan.hpp tells.
// Packed: b is the last sequence whose first tile is j or before it; every lane of
// a wave looks at one of 64. A tile of no sequence gets an i behind every end.
template <typename P>
__device__ __forceinline__ void tile_of(const P& p, int64_t j, int tile, int& b, int& i) {
  if (!p.cu) {
    const int per = (p.seqlen + tile - 1) / tile;
    b = (int)(j / per);
    i = (int)(j - (int64_t)b * per);
    return;
  }
  const int lane = threadIdx.x & 63;
  int from = 0, n = p.batch;  // the sequences among which it is
  auto begun = [&](int s) { return min(max(p.cu[s], 0), p.total) / tile + (int64_t)s <= j; };
  while (n > 64) {
    const int step = (n + 63) / 64, end = from + n;
    const int hits = __popcll(__ballot(lane * step < n && begun(from + lane * step)));
    from += max(hits - 1, 0) * step;
    n = min(step, end - from);
  }
  const int hits = __popcll(__ballot(lane < n && begun(from + lane)));
  b = from + max(hits, 1) - 1;
  i = (int)j - (min(max(uniform_i(p.cu[b]), 0), p.total) / tile + b);
  if (i < 0 || i > p.total / tile) i = p.total / tile + 1;
}

// exp(x) from the hardware's exp2 (about 1 ulp) with what the product x log2 e loses of
// the exponent put back: 2^t (1 + r ln 2), t + r = x log2 e. Below -120 it is 0, above
// 88.72 infinity; NaN stays.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float hi = 1.442695041f, lo = 1.925963e-8f;  // log2 e in two parts
  const float y = x < -120.f ? -120.f : x;
  const float t = y * hi, r = fmaf(y, lo, fmaf(y, hi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return x > 88.72f ? __builtin_inff() : fmaf(e * 0.6931471806f, r, e);
}
// 1 / (1 + exp(-x)): the hardware's reciprocal with one step of Newton's
__device__ __forceinline__ float sigmoid_of(float x, float) {
  const float d = 1.f + exp_f32(-x), y = __builtin_amdgcn_rcpf(d);
  return x < -88.f ? 0.f : fmaf(fmaf(-d, y, 1.f), y, y);
}
// bf16 tensors: the hardware's exp2 and reciprocal, about 1 ulp each
__device__ __forceinline__ float sigmoid_of(float x, bf16) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

// Factor a = exp(la) of a token and 1 - a^2. Near 1 the sum 1 + (a - 1) with a - 1
// from its series: the factor is then off by half a step and not biased, so a
// thousand tokens' product stays good, and 1 - a^2 = (1 - a)(1 + a) has no
// cancellation. bf16 tensors take the series to |la| = 1/32, four terms (1e-8 of a
// - 1), fp32 ones to 1/4, seven (2e-9); beyond it a - 1 is large enough for what a's
// own rounding leaves of it.
template <typename T>
constexpr float kNear = sizeof(T) == 4 ? 0.25f : 0.03125f;
template <typename T>
__device__ __forceinline__ float near_minus_1(float la) {  // exp(la) - 1
  float p;
  if constexpr (sizeof(T) == 4) {
    p = 1.f / 5040;
    p = fmaf(p, la, 1.f / 720);
    p = fmaf(p, la, 1.f / 120);
    p = fmaf(p, la, 1.f / 24);
  } else {
    p = 1.f / 24;
  }
  p = fmaf(p, la, 1.f / 6);
  p = fmaf(p, la, 0.5f);
  return fmaf(p, la, 1.f) * la;
}
template <typename T>
__device__ __forceinline__ void factor(float la, float& a, float& left) {
  const float p = near_minus_1<T>(la);
  const float e = sizeof(T) == 4 ? exp_f32(la) : __builtin_amdgcn_exp2f(1.4426950408889634f * la);
  const bool near = fabsf(la) < kNear<T>;
  a = near ? 1.f + p : e;
  left = near ? -p * (2.f + p) : fmaf(-e, e, 1.f);
}
// 1 - a^2 once more, of a token whose factor is known
template <typename T>
__device__ __forceinline__ float left_of(float la, float a) {
  const float p = near_minus_1<T>(la);
  return fabsf(la) < kNear<T> ? -p * (2.f + p) : fmaf(-a, a, 1.f);
}

// A workgroup's tile and channels. Where tiles hand a state on, a workgroup takes
// them by a ticket, so that whoever it waits for holds a lower one and runs already.
// One counter for all of a launch would serialise its workgroups, so each has one of
// up to 16 for its own run of neighbouring channel groups. Workgroups go round the 8 XCDs,
// so the queues of an XCD get neighbouring runs too: what its workgroups ask for at one
// time are long pieces of a row. Tiles of a queue run along time first, the sequences of a
// batch side by side (reversed in the backward).
// Measured, forward in us, with 32 queues of groups 32 apart, then runs on 64 / 32 / 16 /
// 8 queues: 2 x 8192 x 4096 128, 124 / 119 / 115 / 117; 1 x 16384 x 8192 238, 209 / 202 /
// 202 / 197; 2 x 8192 x 5120 133, 139 / 133 / 137 / 139; 2 x 4096 x 6000 105, 103 / 95 / 95 / 96.
struct ScanQueues {
  int groups, each, queues;  // channel groups, those of a queue, queues
};
__host__ __device__ inline ScanQueues queues_of(int width) {
  ScanQueues q;
  q.groups = (width + kScanChannels - 1) / kScanChannels;
  q.each = (q.groups + kScanQueues - 1) / kScanQueues;
  q.queues = (q.groups + q.each - 1) / q.each;
  return q;
}
// The control word of a call without a launch that clears it.
template <typename P>
__device__ __forceinline__ void clear_errors(const P& p) {
  if (!p.hand && !p.cu && !p.keep_error && blockIdx.x == 0 && threadIdx.x < 2) p.ctrl[threadIdx.x] = 0;
}
struct Place {
  int group, b, i;     // channel group, sequence, tile of it
  int64_t tile;        // its number
  bool any;
};
template <bool BACK, typename P>
__device__ __forceinline__ Place place_of(const P& p, int tile) {
  __shared__ int s_ticket;
  const ScanQueues q = queues_of(p.width);
  const int queue = blockIdx.x % q.queues;
  int ticket = blockIdx.x / q.queues;
  if (p.hand) {
    if (threadIdx.x == 0) s_ticket = atomicAdd(p.ctrl + 16 * (1 + queue), 1);
    __syncthreads();
    ticket = uniform_i(s_ticket);
  }
  Place at;
  const int run = q.queues % 8 ? queue : queue % 8 * (q.queues / 8) + queue / 8;
  at.group = run * q.each + ticket % q.each;
  int j = ticket / q.each;
  if (BACK) j = p.tiles - 1 - j;
  if (p.cu) {
    tile_of(p, j, tile, at.b, at.i);
    at.tile = j;
  } else {
    at.b = j % p.batch;
    at.i = j / p.batch;
    at.tile = (int64_t)at.b * (p.tiles / p.batch) + at.i;
  }
  at.any = at.group < q.groups;
  return at;
}
inline unsigned scan_grid(const ScanParams& p) {
  const ScanQueues q = queues_of(p.width);
  return (unsigned)p.tiles * q.queues * q.each;
}

// A word that hands a value on: the value and a mark, in one store and one load, so
// that nothing else has to be ordered around them. Agent scope: workgroups of other
// XCDs, behind other L2s, see it.
__device__ __forceinline__ void hand_on(uint64_t* word, float x) {
  __hip_atomic_store(word, (uint64_t)__float_as_uint(x) | 1ull << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits until the word is there, in every lane of the wave that asks.
__device__ __forceinline__ float take_over(const uint64_t* word, bool asks, int* ctrl) {
  constexpr int kSpinLimit = 1 << 21;  // more than a second
  uint64_t w = 0;
  for (int spins = 0;; ++spins) {
    if (asks) w = __hip_atomic_load(const_cast<uint64_t*>(word), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__all(!asks || (w >> 32))) break;
    // after an error (bounds that do not follow each other among them) nobody may come
    if (spins % 256 == 255 && __hip_atomic_load(ctrl + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0) break;
    if (spins > kSpinLimit) {
      atomicOr(ctrl + 1, 1);
      break;
    }
  }
  return __uint_as_float((uint32_t)w);
}

// A factor of 0 forgets what was there, NaN and infinity too.
__device__ __forceinline__ float step_or_forget(float a, float h, float u) { return a == 0.f ? u : fmaf(a, h, u); }

// Products of factors. Only a token's own factor of 0 forgets: a product of others that is
// no normal number in 32 bits has to keep a state that is NaN or infinite, and one that is
// 0 or far from 1, whatever stood beside it. So a product is one float where that is a
// normal number, 0 where a token among its own forgot (whatever the other factors were),
// and else -m with an exponent e beside it: m 2^e, m in [1/2, 1), infinity or NaN.
struct Product {
  float m;
  int e;  // meant where m < 0
};
__device__ __forceinline__ bool is_normal(float a) { return a >= 0x1p-126f && a < __builtin_inff(); }
__device__ __forceinline__ float step_over(Product a, float h, float u) {
  const float far = __builtin_ldexpf(-a.m * h, a.e) + u;
  return a.m < 0.f ? far : step_or_forget(a.m, h, u);
}
// The same with the exponent in memory, where it is read only if it is meant.
__device__ __forceinline__ float step_over(float m, const int* e, float h, float u) {
  float y = fmaf(m, h, u);
  if (m <= 0.f) y = m == 0.f ? u : __builtin_ldexpf(-m * h, *e) + u;
  return y;
}
// How such a product grows: m 2^e with m >= 0, from 1. By a factor that is not 0, and by
// the product of some.
struct Growing {
  float m = 1.f;
  int e = 0;
  __device__ __forceinline__ void by(float a) {
    const float q = m * a;
    m = __builtin_amdgcn_frexp_mantf(q);
    e += __builtin_amdgcn_frexp_expf(q);
  }
  __device__ __forceinline__ void by(Product a) {
    const bool none = m == 0.f || a.m == 0.f;
    by(fabsf(a.m));
    e += a.m < 0.f ? a.e : 0;
    if (none) *this = {0.f, 0};
  }
  __device__ __forceinline__ Product product() const { return {-m, e}; }
};

}  // namespace ret
