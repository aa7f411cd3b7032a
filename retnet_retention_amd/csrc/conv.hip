// Short causal convolution along a sequence, a filter of K taps a channel:
//     z_t = bias + sum_j w_j x_(t-K+1+j),   y = z, or z sigmoid(z),
// with the K - 1 inputs before the first token from a carried state (or 0). Its
// gradients, dz = dy swish'(z):
//     dx_t = sum_j w_j dz_(t+K-1-j),   dw_j = sum_t dz_t x_(t-K+1+j),   dbias = sum dz.
// Bound by memory: a wave holds 64 V channels of a tile's tokens and the K - 1 rows
// beside it, so each row is read once but for those.
// Measured in bf16, 4 taps with bias and swish, kernel alone: forward 2 x 8192 x 12288 151 us
// to 154 (5.2 TB/s; a copy reaches 5.07; its stores past the caches were 6 us faster, but then whoever
// reads the result next takes 13 us longer), 2 x 8192 x 6000 79 us (5.0 TB/s); backward 4 x
// 2048 x 7680 85 us (4.5 TB/s) and 5.4 for the sums, with the SIMDs computing in 68 % of their
// cycles, 2 x 8192 x 6000 147 us (4.0 TB/s). fp32, 2 x 8192 x 2048: 49 us (5.5 TB/s) and 90 (4.5).
#include "norms.hpp"
#include "scan_common.hpp"

namespace ret {

constexpr int kConvRows = 32;               // tokens of a wave
constexpr int kConvTile = 4 * kConvRows;    // ... and of a workgroup

// Inputs of a sequence with its state before them: index t, t < 0 in the state, t at
// or behind the end the last one's (never used).
template <typename T, int K, int V>
struct ConvLine {
  const T *x, *state;
  int64_t x_stride;
  int width, len, c;
  __device__ __forceinline__ ConvLine(const ConvParams& p, int b, int tok0, int len_, int c_)
      : x(reinterpret_cast<const T*>(p.x) + tok0 * p.x_stride),
        state(p.state_in ? reinterpret_cast<const T*>(p.state_in) + (int64_t)b * (K - 1) * p.width : nullptr),
        x_stride(p.x_stride), width(p.width), len(len_), c(c_) {}
  __device__ __forceinline__ lane_raw<T, V> token(int t) const {
    return lane_load<T, V>(x + min(t, len - 1) * x_stride, c);
  }
  __device__ __forceinline__ lane_raw<T, V> at(int t) const {
    if (t >= 0) return token(t);
    return state ? lane_load<T, V>(state + (int64_t)(K - 1 + t) * width, c) : lane_raw<T, V>{};
  }
};

// The piece of work, a tile's `groups` channel groups one after the other, of this
// workgroup. Workgroups go round the 8 XCDs; of each 8 s of them an XCD's s, some eighth of
// a tile's row, take neighbouring pieces. Forward and backward in us, taken as they come and
// so: 2 x 8192 x 12288 168 / 279 and 153 / 278, 2 x 8192 x 6000 94 / 157 and 83 / 146, 2 x 8192
// x 5120 72 / 115 and 65 / 112, 2 x 8192 x 4096 44 / 76 and 44 / 78.
__device__ __forceinline__ unsigned piece_of(int groups) {
  const unsigned s = (groups + 7) / 8, at = blockIdx.x % (8 * s), first = blockIdx.x - at;
  return first + 8 * s <= gridDim.x ? first + at % 8 * s + at / 8 : blockIdx.x;
}

template <typename T, int K, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p) {
  constexpr int L = kConvRows;
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int groups = (p.width + 64 * V - 1) / (64 * V);
  int b, i, tok0, len;
  const unsigned piece = piece_of(groups);
  tile_of(p, piece / groups, kConvTile, b, i);
  span_of(p, b, tok0, len);
  const int c = (piece % groups * 64 + lane) * V;
  const int t0 = i * kConvTile + wave * L;
  const bool ends = p.state_out && i == 0 && wave == 0;  // reads the old state, and so writes the new one
  if (c >= p.width || (t0 >= len && !ends)) return;
  const ConvLine<T, K, V> line(p, b, tok0, len, c);
  lane_raw<T, V> last[K - 1];
  if (ends) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) last[j] = line.at(len - (K - 1) + j);
  }
  if (t0 < len) {
    lane_raw<T, V> r[L + K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j] = line.at(t0 - (K - 1) + j);
#pragma unroll
    for (int j = K - 1; j < L + K - 1; ++j) r[j] = line.token(t0 - (K - 1) + j);
    float w[V][K], bias[V], x[K][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      bias[e] = p.bias ? p.bias[c + e] : 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[e][j] = p.weight[(int64_t)(c + e) * K + j];
    }
    T* o = reinterpret_cast<T*>(p.o) + ((int64_t)tok0 + t0) * p.width;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Lane<T, V>::get(r[j], x[j]);
#pragma unroll
    for (int j = 0; j < L; ++j) {
      Lane<T, V>::get(r[j + K - 1], x[(j + K - 1) % K]);
      float z[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        z[e] = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k) z[e] = fmaf(w[e][k], x[(j + k) % K][e], z[e]);
        if (p.swish) z[e] *= sigmoid_of(z[e], T());
      }
      if (t0 + j < len) lane_store<T, V>(o + (int64_t)j * p.width, c, z);
    }
  }
  if (ends) {
    T* out = reinterpret_cast<T*>(p.state_out) + (int64_t)b * (K - 1) * p.width;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) *reinterpret_cast<lane_raw<T, V>*>(out + (int64_t)j * p.width + c) = last[j];
  }
}

// A wave walks `p.rows` tokens, kConvStep at a time, the next ones on their way from
// memory; what it carries are the last K - 1 inputs and dz. It looks K - 1 tokens past
// its own for the dx of its last ones. dx goes past the caches, but not where rows end inside
// a line of 128 bytes, whose parts two workgroups write. Past them and through them, a call
// with x in memory and dout just written, that call with a matrix product that reads dx, and
// calls one after the other: 2 x 8192 x 6000 163 / 326 / 151 us and 133 / 298 / 145, 4 x 2048 x
// 7680 81 / 209 / 84 and 82 / 212 / 88, 2 x 8192 x 4096 87 / 193 / 94 and 85 / 192 / 96, 2 x
// 8192 x 12288 278 / 575 / 255 and 267 / 565 / 261.
constexpr int kConvStep = 8;

template <typename T, int K, int V>
__global__ __launch_bounds__(256, 4) void conv_bwd_kernel(ConvParams p) {
  constexpr int S = kConvStep, H = K - 1;
  __shared__ float s_sum[4][K + 1][64 * V];
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int groups = (p.width + 64 * V - 1) / (64 * V);
  const unsigned piece = piece_of(groups);
  const int64_t block = piece / groups;
  int b, i, tok0, len;
  tile_of(p, block, 4 * p.rows, b, i);
  span_of(p, b, tok0, len);
  const int at = (piece % groups * 64 + lane) * V, c = min(at, p.width - V);
  const bool inside = at < p.width;
  const int t0 = (4 * i + wave) * p.rows;
  const bool begins = i == 0 && wave == 0;
  T* dx = reinterpret_cast<T*>(p.dx);
  // rows before the first sequence and behind the last have gradient 0
  auto clear = [&](int from, int to) {
    const float zero[V] = {};
    for (int t = from + wave; t < to && inside; t += 4) lane_store<T, V>(dx + (int64_t)t * p.width, c, zero);
  };
  if (p.cu && i == 0 && b == 0) clear(0, tok0);
  if (p.cu && i == 0 && b == p.batch - 1) clear(tok0 + len, p.total);
  dx += (int64_t)tok0 * p.width;
  const int64_t held = (int64_t)b * H * p.width;
  const T* after = p.d_state_out ? reinterpret_cast<const T*>(p.d_state_out) + held : nullptr;
  // what the state behind the last token adds to index s
  auto add_after = [&](int s, float* d) {
    const int j = s + H - len;
    if (after && j >= 0) {
      float y[V];
      Lane<T, V>::get(lane_load<T, V>(after + (int64_t)j * p.width, c), y);
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] += y[e];
    }
  };
  auto put_state = [&](int s, float* d) {
    add_after(s, d);
    if (inside) lane_store<T, V>(reinterpret_cast<T*>(p.d_state_in) + held + (int64_t)(H + s) * p.width, c, d);
  };
  float w[V][K], bias[V], sum[K + 1][V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    bias[e] = p.bias ? p.bias[c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[e][j] = p.weight[(int64_t)(c + e) * K + j];
#pragma unroll
    for (int j = 0; j < K + 1; ++j) sum[j][e] = 0.f;
  }
  if (t0 < len) {
    const ConvLine<T, K, V> line(p, b, tok0, len, c);
    const T* dout = reinterpret_cast<const T*>(p.dout) + (int64_t)tok0 * p.width;
    const int end = min(t0 + p.rows + H, len);  // tokens that are looked at
    lane_raw<T, V> nx[S], nd[S];
    const int rows = min(p.rows + H, len - t0);
    const Rows<T, V> xs(line.x + t0 * p.x_stride, p.x_stride, rows, p.width, 0, c);
    const Rows<T, V> ds(dout + (int64_t)t0 * p.width, p.width, rows, p.width, 0, c);
    const Rows<T, V> to(dx + (int64_t)t0 * p.width, p.width, rows, p.width, 0, c);
    const bool lines = (uint32_t)p.width * (uint32_t)sizeof(T) % 128 == 0;
    auto ask = [&](int t) {
      const int from = t - t0;
      if (from + S <= rows) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          nx[j] = xs.load(from + j);
          nd[j] = ds.load(from + j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          nx[j] = xs.load_if(from + j);
          nd[j] = ds.load_if(from + j);
        }
      }
    };
    ask(t0);
    float x[S + H][V], dz[S + H][V];  // the first H: of the tokens before
#pragma unroll
    for (int j = 0; j < H; ++j) {
      Lane<T, V>::get(line.at(t0 - H + j), x[j]);
#pragma unroll
      for (int e = 0; e < V; ++e) dz[j][e] = 0.f;
    }
    for (int t = t0; t < t0 + p.rows + H && t - H < len; t += S) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        Lane<T, V>::get(nx[j], x[H + j]);
        Lane<T, V>::get(nd[j], dz[H + j]);
      }
      if (t + S < end) ask(t + S);
      auto step = [&](auto whole, auto stream) {
        // whole: every token is one of the wave's own, and none of the last H of the sequence
        constexpr bool FULL = decltype(whole)::value;
        constexpr int POLICY = decltype(stream)::value ? kStreamed : 0;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const bool there = FULL || t + j < end, own = FULL || (there && t + j < t0 + p.rows);
          float out[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float& d = dz[H + j][e];
            if (p.swish) {
              float z = bias[e];
#pragma unroll
              for (int k = 0; k < K; ++k) z = fmaf(w[e][k], x[j + k][e], z);
              const float s = sigmoid_of(z, T());
              d *= s * fmaf(z, 1.f - s, 1.f);
            }
            if (!there) d = 0.f;
            if (own) {
#pragma unroll
              for (int k = 0; k < K; ++k) sum[k][e] = fmaf(d, x[j + k][e], sum[k][e]);
              sum[K][e] += d;
            }
            out[e] = w[e][0] * d;
#pragma unroll
            for (int k = 1; k < K; ++k) out[e] = fmaf(w[e][k], dz[H + j - k][e], out[e]);
          }
          const int s = t + j - H;
          if (FULL || s >= t0) {
            if (FULL || (s < len && s < t0 + p.rows)) {
              if (!FULL) add_after(s, out);
              if (inside) to.template store<POLICY>(s - t0, out);
            }
          } else if (begins && p.d_state_in) {
            put_state(s, out);
          }
        }
      };
      if (t > t0 && t + S <= min(t0 + p.rows, len)) {
        if (lines)
          step(std::true_type(), std::true_type());
        else
          step(std::true_type(), std::false_type());
      } else {
        step(std::false_type(), std::false_type());
      }
#pragma unroll
      for (int j = 0; j < H; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[j][e] = x[S + j][e];
          dz[j][e] = dz[S + j][e];
        }
    }
  } else if (begins && len == 0 && p.d_state_in) {
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float d[V] = {};
      put_state(j - H, d);
    }
  }
#pragma unroll
  for (int j = 0; j < K + 1; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) s_sum[wave][j][lane * V + e] = sum[j][e];
  __syncthreads();
  for (int k = wave; k < K + 1; k += 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) s += s_sum[v][k][lane * V + e];
      if (inside) p.partial[(block * (K + 1) + k) * p.width + c + e] = s;
    }
  }
}

// The weights' gradients from the workgroups' sums: 64 channels a workgroup, 16
// strands of sums added in order. blockIdx.y: the tap, or behind the last the bias.
template <int K>
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* partial, int64_t blocks, int width, float* dweight,
                                                        float* dbias) {
  __shared__ float s[16][64];
  const int k = blockIdx.y, lane = threadIdx.x & 63, c = blockIdx.x * 64 + lane, strand = threadIdx.x >> 6;
  if (k == K && !dbias) return;
  float x = 0.f;
  if (c < width)
#pragma unroll 8
    for (int64_t i = strand; i < blocks; i += 16) x += partial[(i * (K + 1) + k) * width + c];
  s[strand][lane] = x;
  __syncthreads();
  if (strand == 0 && c < width) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += s[i][lane];
    (k < K ? dweight[(int64_t)c * K + k] : dbias[c]) = x;
  }
}

// Tokens of a wave in the backward: many, as each looks K - 1 past its own on both
// sides and leaves a row of sums, but at least 4096 waves of 128 channels, 16 a CU.
// With 16 / 32 / 64 / 128: 4 x 2048 x 7680 109 / 86 / 75 / 72 us, 8 x 2048 x 2048 54 / 50 /
// 45 / 45, 1 x 8192 x 1024 19 / 19 / 22 / 30.
int conv_bwd_rows(int64_t tokens, int width) {
  const int64_t groups = (width + 127) / 128;
  int rows = 128;
  while (rows > 16 && tokens / rows * groups < 4096) rows /= 2;
  return rows;
}
int64_t conv_bwd_blocks(int batch, int seqlen, int width, bool packed, int64_t total) {
  const int64_t tokens = packed ? total : (int64_t)batch * seqlen;
  return tile_count(batch, seqlen, packed, total, 4 * conv_bwd_rows(tokens, width));
}

// Pairs of bf16 channels where they are aligned in every row.
template <typename T, int K, typename F>
static hipError_t with_lanes(const ConvParams& p, F&& f) {
  if (sizeof(T) == 2 && p.width % 2 == 0 && pairs_aligned(p.x, p.x_stride, 2))
    return f(std::integral_constant<int, sizeof(T) == 2 ? 2 : 1>());
  return f(std::integral_constant<int, 1>());
}
template <typename T, int K>
static hipError_t launch_conv_fwd_k(const ConvParams& p, hipStream_t stream) {
  return with_lanes<T, K>(p, [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int64_t n = tile_count(p.batch, p.seqlen, p.cu, p.total, kConvTile) * ((p.width + 64 * V - 1) / (64 * V));
    hipLaunchKernelGGL((conv_fwd_kernel<T, K, V>), dim3((unsigned)n), dim3(256), 0, stream, p);
    return hipGetLastError();
  });
}
template <typename T, int K>
static hipError_t launch_conv_bwd_k(ConvParams p, hipStream_t stream) {
  const int64_t tiles = conv_bwd_blocks(p.batch, p.seqlen, p.width, p.cu, p.total);
  p.rows = conv_bwd_rows(p.total, p.width);
  const hipError_t e = with_lanes<T, K>(p, [&](auto v) {
    constexpr int V = decltype(v)::value;
    const int64_t n = tiles * ((p.width + 64 * V - 1) / (64 * V));
    hipLaunchKernelGGL((conv_bwd_kernel<T, K, V>), dim3((unsigned)n), dim3(256), 0, stream, p);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((conv_sum_kernel<K>), dim3((p.width + 63) / 64, K + 1), dim3(1024), 0, stream, p.partial, tiles,
                     p.width, p.dweight, p.dbias);
  return hipGetLastError();
}
template <typename T>
static hipError_t launch_conv(const ConvParams& p, int taps, bool grad, hipStream_t s) {
  switch (taps) {
    case 2: return grad ? launch_conv_bwd_k<T, 2>(p, s) : launch_conv_fwd_k<T, 2>(p, s);
    case 3: return grad ? launch_conv_bwd_k<T, 3>(p, s) : launch_conv_fwd_k<T, 3>(p, s);
    case 4: return grad ? launch_conv_bwd_k<T, 4>(p, s) : launch_conv_fwd_k<T, 4>(p, s);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_conv_fwd(const ConvParams& p, int taps, int dtype, hipStream_t stream) {
  if (p.cu) {
    const hipError_t e = launch_check_bounds(p.cu, p.batch, p.total, p.ctrl, stream);
    if (e != hipSuccess) return e;
  }
  return dtype == 1 ? launch_conv<bf16>(p, taps, false, stream) : launch_conv<float>(p, taps, false, stream);
}
hipError_t launch_conv_bwd(const ConvParams& p, int taps, int dtype, hipStream_t stream) {
  if (p.cu) {
    const hipError_t e = launch_check_bounds(p.cu, p.batch, p.total, p.ctrl, stream);
    if (e != hipSuccess) return e;
  }
  return dtype == 1 ? launch_conv<bf16>(p, taps, true, stream) : launch_conv<float>(p, taps, true, stream);
}

}  // namespace ret
