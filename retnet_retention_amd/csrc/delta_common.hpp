// Device helpers of the delta-rule kernels.
#pragma once

#include "common.hpp"
#include "delta.hpp"

namespace ret {

constexpr int kB = kDeltaBlock;

// Logarithmic decays below this are a reset (exp gives 0 either way); the
// bound keeps differences of sums finite.
constexpr float kMinLogDecay = -1e5f;
constexpr float kZeroLogDecay = -104.f;  // exp of less is 0 in 32 bits (2^-149 = exp(-103.3))

// An fp32 operand of the matrix cores: for bf16 tensors as the sum of two
// bf16 values (the rounded value and the rounded rest, together 16 bits or
// more), for fp32 tensors as it is. The state, the inverse T and the written
// values V' feed each other from block to block, so one bf16 rounding each
// (2^-9) would reach the fp32 state a call returns; with the rest (2^-18 a
// product) the state is within 5e-6 over 8192 tokens. A third value
// would cost half as many products again on the way from block to block.
template <typename T> struct Planes;
template <> struct Planes<bf16> { static constexpr int N = 2; };
template <> struct Planes<float> { static constexpr int N = 1; };

template <typename T> struct Split { frag_t<T> f[Planes<T>::N]; };

// elements 8 SL .. 8 SL + 7 of a 32x32 accumulator as an operand
template <int SL>
__device__ __forceinline__ Split<bf16> split_acc(const f32x16& c, bf16*) {
  Split<bf16> s;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bf16 hi = (bf16)c[8 * SL + j];
    s.f[0][j] = hi;
    s.f[1][j] = (bf16)(c[8 * SL + j] - (float)hi);
  }
  return s;
}
template <int SL>
__device__ __forceinline__ Split<float> split_acc(const f32x16& c, float*) {
  Split<float> s;
#pragma unroll
  for (int j = 0; j < 8; ++j) s.f[0][j] = c[8 * SL + j];
  return s;
}

// The 64 x 64 matrices T, M and P and what they multiply (X, dV') pass every
// value on. The forward takes them as two values, the backward as three (24 bits):
// with two, d beta (dv . V' / beta^2, both factors through T) was 8e-6 off, with
// three 5e-6, for 3 to 7% of the call.
template <typename T, bool GRAD> struct MatPlanes {
  static constexpr int N = sizeof(T) == 4 ? 1 : GRAD ? 3 : 2;
};

// a * b, both in planes: products of rests smaller than 2^-24 are left out
template <int NA, int NB, typename F>
__device__ __forceinline__ f32x4 mma_planes(const F (&a)[NA], const F (&b)[NB], f32x4 c) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j <= 2) c = mma(a[i], b[j], c);
  return c;
}

// the key column within 32 of position n in that order
__device__ __forceinline__ constexpr int state_col(int n) {
  return (n & 16) + 4 * ((((n >> 2) & 1) << 1) | ((n >> 3) & 1)) + (n & 3);
}
// the same fragment of a tile filled by direct loads (rows: value columns)
template <typename TL>
__device__ __forceinline__ bf16x8 state_tile_col8(const char* m, int k0, int n0, int lane, bf16*) {
  const int grp = lane >> 4, t = lane & 15, h = grp >> 1;
  const char* p = m + TL::off(k0 + 4 * h + (t >> 2), n0 + 16 * (grp & 1) + state_col(4 * (t & 3)));
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + TL::row_step(8)));
  typedef short i16x8 __attribute__((ext_vector_type(8)));
  const i16x8 w = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, w);
}
template <typename TL>
__device__ __forceinline__ f32x8 state_tile_col8(const char* m, int k0, int n0, int lane, float*) {
  const int h = lane >> 5, col = n0 + state_col(lane & 31);
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = *reinterpret_cast<const float*>(m + TL::off(k0 + 4 * h + j, col));
    f[4 + j] = *reinterpret_cast<const float*>(m + TL::off(k0 + 8 + 4 * h + j, col));
  }
  return f;
}

// ---------------------------------------------------------------------------
// Operands laid out by delta_prep_kernel in the order the lanes take them, 64 x
// 8 elements a fragment: a wave's load of one is 1 or 2 KiB in a row (rows of
// the tensors are far apart, and a lane's 8 elements of its own row cost the
// caches a request each).
//   keys of a block and key head: [D / 16][2][64 lanes]   (32x32 row fragments)
//   the same by columns (and of queries, backward): [D / 32][4][64 lanes]
//   queries:                      [4][D / 32][64 lanes]   (16x16 row fragments)
//   64 x 64 matrices, per plane:  [4][2][64 lanes]        (16x16 row fragments)
// ---------------------------------------------------------------------------
constexpr int kFrag = 64 * 8;
__device__ __forceinline__ constexpr int key_frag(int ks, int rt) { return (2 * ks + rt) * kFrag; }
__device__ __forceinline__ constexpr int column_frag(int tile, int ks) { return (4 * tile + ks) * kFrag; }
template <int D>
__device__ __forceinline__ constexpr int query_frag(int rb, int ks) { return (rb * (D / 32) + ks) * kFrag; }
__device__ __forceinline__ constexpr int mat_frag(int plane, int rb, int ks) { return ((plane * 4 + rb) * 2 + ks) * kFrag; }

// Rows of sequence b (clamped into the tensors for packed bounds) and the
// number of its first block over the batch.
__device__ __forceinline__ void seq_span(const DeltaParams& p, int b, int64_t& tok0, int& len, int& base) {
  if (p.cu) {
    int t0, n;
    packed_span(p.cu, b, p.total, p.seqlen, t0, n);
    tok0 = t0;
    len = n;
    base = t0 / kB + b;
  } else {
    tok0 = (int64_t)b * p.seqlen;
    len = p.seqlen;
    base = b * p.blocks_max;
  }
}

// Accumulator rows of the state. A wave's state tile t (32 rows) keeps the key
// row 16 s + 8 h + j in the accumulator row of lane half h that the matrix
// cores take as element j of contraction step s, so an accumulator is an
// operand as it stands and the operand that meets it is 8 consecutive
// elements of a token's row.
//   key row within the tile of accumulator element i, half h:
__device__ __forceinline__ constexpr int state_row(int i, int h) { return 16 * (i / 8) + 8 * h + (i % 8); }

// ---------------------------------------------------------------------------
// How a workgroup holds the state of SL value columns: four waves, wave w the
// key rows 32 TPW (w % RG) .. of the columns 32 (w / RG) .. + 31, TPW tiles of
// 32 x 32. Another four waves of the workgroup take what is not on the way
// from one block's state to the next.
// ---------------------------------------------------------------------------
template <typename T, int D>
struct ChainShape {
  static constexpr int TPW = D == 256 ? 2 : 1;
  static constexpr int RG = D == 64 ? 2 : 4;
  static constexpr int CG = 4 / RG;
  static constexpr int KR = 32 * TPW;   // key rows of a wave
  static constexpr int KS = 2 * TPW;    // contraction steps over them
  static constexpr int SL = 32 * CG;    // value columns of a workgroup
  static constexpr int NSL = D / SL;
  static constexpr int CT = 2 * CG;     // 16-column tiles of a wave's quarter of the tokens
  // operand copies [column][token] in LDS: 64 tokens and padding
  static constexpr int PITCH = sizeof(T) == 2 ? 72 : 68;
  static constexpr int OPLANE = SL * PITCH;  // elements of one plane
  static constexpr int OPND = OPLANE * Planes<T>::N;
  // copy of the state [column][key row] in LDS
  static constexpr int SPITCH = D + (sizeof(T) == 2 ? 8 : 4);
  static constexpr int SPLANE = SL * SPITCH;
};

// Column fragment of a row-major LDS array (`pitch` elements a row) as the state
// products take it: tokens k0 .. k0 + 15 (lane half h the tokens k0 + 4h .. + 3
// and k0 + 8 + 4h .. + 3) of the 32 key columns from n0 in the accumulator's
// order: inside 16 columns the groups of four come as 0, 2, 1, 3.
__device__ __forceinline__ bf16x8 state_col8(const bf16* m, int pitch, int k0, int n0, int lane) {
  const int grp = lane >> 4, t = lane & 15, h = grp >> 1;
  const int q = t & 3, cg = ((q & 1) << 1) | (q >> 1);
  const bf16* p = m + (k0 + 4 * h + (t >> 2)) * pitch + n0 + 16 * (grp & 1) + 4 * cg;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 8 * pitch));
  typedef short i16x8 __attribute__((ext_vector_type(8)));
  const i16x8 w = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ f32x8 state_col8(const float* m, int pitch, int k0, int n0, int lane) {
  const int n = lane & 31, h = lane >> 5;
  const int q = (n >> 2) & 3, cg = ((q & 1) << 1) | (q >> 1);
  const float* p = m + (k0 + 4 * h) * pitch + n0 + (n & 16) + 4 * cg + (n & 3);
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = p[j * pitch];
    f[4 + j] = p[(8 + j) * pitch];
  }
  return f;
}

// A value column of a workgroup and its place: the quarter-row products take
// column 32 (ct / 2) + 2 c + ct % 2 as column c of tile ct, so that a lane
// holds neighbouring columns. Copies in LDS keep it in row row_of(ct, c): odd
// tiles in another order, so that 16 columns in a row meet distinct banks
// whichever way they are numbered.
__device__ __forceinline__ constexpr int row_of(int ct, int c) { return 16 * ct + (c ^ ((ct & 1) << 3)); }
__device__ __forceinline__ constexpr int col_place(int n) { return row_of(n & 1, n >> 1); }  // within 32 columns
__device__ __forceinline__ constexpr int col_at(int place) {                                // its inverse
  return 2 * ((place & 15) ^ ((place >> 4) << 3)) + (place >> 4);
}

// Partial products of the waves, [wave][quad of rows][place of column] of 4
// rows each.
__device__ __forceinline__ void put_partial(f32x4* buf, int wave, int rt, const f32x16& acc, int lane) {
  const int n = lane & 31, h = lane >> 5;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    buf[(wave * 16 + 8 * rt + 2 * q + h) * 32 + col_place(n)] =
        f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
}
template <int RG>
__device__ __forceinline__ f32x4 get_partial(const f32x4* buf, int ct, int quad, int c) {
  const f32x4* at = buf + ((ct >> 1) * RG * 16 + quad) * 32 + row_of(ct & 1, c);
  f32x4 s = *at;
#pragma unroll
  for (int r = 1; r < RG; ++r) s += at[r * 512];
  return s;
}

// Four tokens' values of one column into an operand copy, in N planes.
template <int PITCH, int OPLANE, int N>
__device__ __forceinline__ void put_opnd(bf16* m, int row, int at, f32x4 x) {
#pragma unroll
  for (int pl = 0; pl < N; ++pl) {
    bf16x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = (bf16)x[i];
      x[i] -= (float)y[i];
    }
    *reinterpret_cast<bf16x4*>(m + pl * OPLANE + row * PITCH + at) = y;
  }
}
template <int PITCH, int OPLANE, int N>
__device__ __forceinline__ void put_opnd(float* m, int row, int at, const f32x4& x) {
  *reinterpret_cast<f32x4*>(m + row * PITCH + at) = x;
}

// rows of four within 16 tokens as the state products take them: a lane half
// reads its two quads side by side
__device__ __forceinline__ constexpr int quad_place(int g) { return 4 * (((g & 1) << 1) | (g >> 1)); }

// ---------------------------------------------------------------------------
// Reads and writes through a buffer descriptor whose end is the end of what
// exists: rows behind it read as zero and are not written, without a branch.
// ---------------------------------------------------------------------------
// `at` is the part of the offset that is the same in all lanes (a scalar: a
// vector register for each constant would cost more registers than the data).
__device__ __forceinline__ u32x4b raw_load16(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b128(rs, off, at, 0);
}
__device__ __forceinline__ bf16x8 buf_frag(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at, bf16*) {
  return __builtin_bit_cast(bf16x8, raw_load16(rs, off, at));
}
__device__ __forceinline__ f32x8 buf_frag(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at, float*) {
  const f32x4 a = __builtin_bit_cast(f32x4, raw_load16(rs, off, at));
  const f32x4 b = __builtin_bit_cast(f32x4, raw_load16(rs, off + 16, at));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x4 buf_f4(__amdgpu_buffer_rsrc_t rs, uint32_t off, uint32_t at) {
  return __builtin_bit_cast(f32x4, raw_load16(rs, off, at));
}
// two neighbouring elements
typedef uint32_t u32x2b __attribute__((ext_vector_type(2)));
template <typename T> struct PairOf;
template <> struct PairOf<bf16> {
  uint32_t w;
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(e ? w & 0xffff0000u : w << 16); }
};
template <> struct PairOf<float> {
  u32x2b w;
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(w[e]); }
};
__device__ __forceinline__ PairOf<bf16> buf_pair(__amdgpu_buffer_rsrc_t rs, uint32_t off, bf16*) {
  return PairOf<bf16>{__builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0)};
}
__device__ __forceinline__ PairOf<float> buf_pair(__amdgpu_buffer_rsrc_t rs, uint32_t off, float*) {
  return PairOf<float>{__builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0)};
}
__device__ __forceinline__ void buf_put_pair(__amdgpu_buffer_rsrc_t rs, uint32_t off, float a, float b, bf16*) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 x = {(bf16)a, (bf16)b};
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), rs, off, 0, 0);
}
__device__ __forceinline__ void buf_put_pair(__amdgpu_buffer_rsrc_t rs, uint32_t off, float a, float b, float*) {
  __builtin_amdgcn_raw_buffer_store_b64(u32x2b{__float_as_uint(a), __float_as_uint(b)}, rs, off, 0, 0);
}

__device__ __forceinline__ int xcd_swizzle(int id, int total) {
  // workgroups go round the 8 XCDs; neighbours in the result share an XCD's L2
  return total % 8 == 0 ? (id & 7) * (total >> 3) + (id >> 3) : id;
}

}  // namespace ret
