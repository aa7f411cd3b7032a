// Device helpers of the delta-rule kernels.
#pragma once

#include "common.hpp"
#include "delta.hpp"

namespace ret {

constexpr int kB = kDeltaBlock;

// Logarithmic decays below this are a reset (exp gives 0 either way); the
// bound keeps differences of sums finite.
constexpr float kMinLogDecay = -1e5f;

// An fp32 operand of the matrix cores: for bf16 tensors as the sum of two
// bf16 values (the rounded value and the rounded rest, together 16 bits or
// more), for fp32 tensors as it is. The state, the inverse T and the written
// values V' feed each other from block to block, so one bf16 rounding each
// (2^-9) would reach the fp32 state a call returns; with the rest the state
// is within a few 1e-6.
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

// a * b with the products of two roundings' rests left out (2^-18)
template <typename A, typename B, typename C>
__device__ __forceinline__ C mma_split2(const A* a, const B* b, C c, bf16*) {
  c = mma(a[0], b[1], c);
  c = mma(a[1], b[0], c);
  return mma(a[0], b[0], c);
}
template <typename A, typename B, typename C>
__device__ __forceinline__ C mma_split2(const A* a, const B* b, C c, float*) {
  return mma(a[0], b[0], c);
}

// 8 consecutive elements of global memory as a fragment, zero unless `keep`
template <typename T>
__device__ __forceinline__ frag_t<T> global_row8(const T* p, bool keep) {
  if (!keep) return zero_frag<T>();
  return __builtin_bit_cast(frag_t<T>, *reinterpret_cast<const frag_t<T>*>(p));
}

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

// A wave's 64 tokens x KR key columns in LDS, written by rows (8 elements of a
// token's row) and read by columns. 16-byte chunks of a bf16 row are swapped
// within the row by its number, so that 16 rows' writes of one chunk and the
// transposed reads of 4 rows x 4 chunks meet distinct banks.
template <typename T, int KR> struct KeyTile;
template <int KR> struct KeyTile<bf16, KR> {
  static constexpr int BYTES = kB * KR * 2;
  __device__ static __forceinline__ int chunk(int r, int ch) {
    const int f = KR == 64 ? ((((r >> 1) & 1) << 2) | ((r >> 2) & 3)) : ((r >> 2) & 3);
    return r * (KR * 2) + ((ch ^ f) << 4);
  }
  __device__ static __forceinline__ void put(char* t, int r, int col, const bf16x8& x) {
    *reinterpret_cast<bf16x8*>(t + chunk(r, col >> 3)) = x;
  }
  // Column fragment of tokens k0 .. k0 + 15 (k0 a multiple of 16, lane half h
  // the tokens k0 + 4h .. and k0 + 8 + 4h ..) and of the 32 key columns from n0
  // in the accumulator's order: inside 16 columns the groups of four come as
  // 0, 2, 1, 3.
  __device__ static __forceinline__ bf16x8 col(const char* t, int k0, int n0, int lane) {
    const int grp = lane >> 4, m = lane & 15, h = grp >> 1;
    const int q = m & 3, cg = ((q & 1) << 1) | (q >> 1);
    const int c = n0 + 16 * (grp & 1) + 4 * cg, r = k0 + 4 * h + (m >> 2);
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(t + chunk(r, c >> 3) + 2 * (c & 7)));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(t + chunk(r + 8, c >> 3) + 2 * (c & 7)));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    const i16x8 w = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, w);
  }
};
template <int KR> struct KeyTile<float, KR> {
  static constexpr int BYTES = kB * KR * 4;
  __device__ static __forceinline__ void put(char* t, int r, int col, const f32x8& x) {
    f32x4* p = reinterpret_cast<f32x4*>(t + (r * KR + col) * 4);
    p[0] = f32x4{x[0], x[1], x[2], x[3]};
    p[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
  __device__ static __forceinline__ f32x8 col(const char* t, int k0, int n0, int lane) {
    const int n = lane & 31, h = lane >> 5;
    const int q = (n >> 2) & 3, cg = ((q & 1) << 1) | (q >> 1);
    const float* p = reinterpret_cast<const float*>(t) + (k0 + 4 * h) * KR + n0 + (n & 16) + 4 * cg + (n & 3);
    f32x8 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = p[j * KR];
      f[4 + j] = p[(8 + j) * KR];
    }
    return f;
  }
};

// A value column of a workgroup and its place: the quarter-row products take
// column 32 (ct / 2) + 2 c + ct % 2 as column c of tile ct, so that a lane
// holds neighbouring columns; operand copies keep it in row 16 ct + c.
__device__ __forceinline__ constexpr int col_place(int n) { return ((n & 1) << 4) | (n >> 1); }  // within 32 columns

// Partial products of the waves, [wave][quad of rows][place of column] of 4
// rows each.
__device__ __forceinline__ void put_partial(f32x4* buf, int wave, const f32x16* acc, int lane) {
  const int n = lane & 31, h = lane >> 5;
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      buf[(wave * 16 + 8 * rt + 2 * q + h) * 32 + col_place(n)] =
          f32x4{acc[rt][4 * q], acc[rt][4 * q + 1], acc[rt][4 * q + 2], acc[rt][4 * q + 3]};
}
template <int RG>
__device__ __forceinline__ f32x4 get_partial(const f32x4* buf, int ct, int quad, int c) {
  f32x4 s = buf[((ct >> 1) * RG * 16 + quad) * 32 + (ct & 1) * 16 + c];
#pragma unroll
  for (int r = 1; r < RG; ++r) s += buf[(((ct >> 1) * RG + r) * 16 + quad) * 32 + (ct & 1) * 16 + c];
  return s;
}

// Four tokens' values of one column into an operand copy, in planes.
template <int PITCH, int OPLANE>
__device__ __forceinline__ void put_opnd(bf16* m, int row, int at, const f32x4& x) {
  bf16x4 hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = (bf16)x[i];
    lo[i] = (bf16)(x[i] - (float)hi[i]);
  }
  *reinterpret_cast<bf16x4*>(m + row * PITCH + at) = hi;
  *reinterpret_cast<bf16x4*>(m + OPLANE + row * PITCH + at) = lo;
}
template <int PITCH, int OPLANE>
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
__device__ __forceinline__ u32x4b raw_load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
}
__device__ __forceinline__ bf16x8 buf_frag(__amdgpu_buffer_rsrc_t rs, uint32_t off, bf16*) {
  return __builtin_bit_cast(bf16x8, raw_load16(rs, off));
}
__device__ __forceinline__ f32x8 buf_frag(__amdgpu_buffer_rsrc_t rs, uint32_t off, float*) {
  const f32x4 a = __builtin_bit_cast(f32x4, raw_load16(rs, off)), b = __builtin_bit_cast(f32x4, raw_load16(rs, off + 16));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x4 buf_f4(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(f32x4, raw_load16(rs, off));
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

// Barrier of the waves' LDS traffic alone: loads and stores of global memory
// stay in flight across it.
__device__ __forceinline__ void lds_barrier() { __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ int xcd_swizzle(int id, int total) {
  // workgroups go round the 8 XCDs; neighbours in the result share an XCD's L2
  return total % 8 == 0 ? (id & 7) * (total >> 3) + (id >> 3) : id;
}

}  // namespace ret
