// Gradients of the norms around a token mixer. With n = norm(x), r its inverse
// deviation and g the gradient of n, the row's gradient is
//     r (g - mean(g) [centred] - n mean(g n));
// the weights' gradients are sums over all rows: a workgroup sums its rows in
// registers, writes one row of sums, and a second launch adds these up in a
// fixed order. Everything the forward formed is formed again from its inputs,
// so one pass reads each tensor once, the next row on its way while one is
// worked on. Head norm: 36 + 5 us for 8192 tokens of 10 heads of 256, bf16 (210
// MB: 5.1 TB/s with the column sums); residual norm: 163 us for 16384 rows of 4096
// with all weights (805 MB: 4.9 TB/s).
#include "norm_rows.hpp"

namespace ret {

// Column sums of one workgroup: its RPB rows of lanes are added in order.
template <typename R>
__device__ __forceinline__ void put_sums(const float* acc, float* out, int width, float* lds) {
  const int l = threadIdx.x % R::LPR, grp = threadIdx.x / R::LPR;
  if constexpr (R::RPB == 1) {
    R::store(out, acc, width, l);
  } else {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R::E; ++j) lds[(grp * R::E + j) * R::LPR + l] = acc[j];
    __syncthreads();
    if (grp == 0) {
      float s[R::E];
#pragma unroll
      for (int j = 0; j < R::E; ++j) {
        s[j] = 0.f;
#pragma unroll
        for (int g = 0; g < R::RPB; ++g) s[j] += lds[(g * R::E + j) * R::LPR + l];
      }
      R::store(out, s, width, l);
    }
  }
}

template <typename T, typename R>
__global__ __launch_bounds__(R::THREADS) void head_norm_bwd_kernel(NormParams p) {
  __shared__ float sh[64];
  __shared__ float lds[R::RPB == 1 ? 1 : R::THREADS * R::E];
  int turn = 0;
  const int l = threadIdx.x % R::LPR;
  float w[R::E], acc[R::E];
  if (p.weight) R::load(w, p.weight, p.width, l);
#pragma unroll
  for (int j = 0; j < R::E; ++j) {
    if (!p.weight) w[j] = 1.f;
    acc[j] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * R::RPB;
  typename R::Raw rx, rd, rg;
  auto ask = [&](int64_t row) {
    const int64_t at = row * p.width;
    const bool keep = row < p.rows;
    R::ask(rx, reinterpret_cast<const T*>(p.x) + at, p.width, l, keep);
    R::ask(rd, reinterpret_cast<const T*>(p.dout) + at, p.width, l, keep);
    if (p.gate) R::ask(rg, reinterpret_cast<const T*>(p.gate) + at, p.width, l, keep);
  };
  ask((int64_t)blockIdx.x * R::RPB + threadIdx.x / R::LPR);
  for (int64_t first = (int64_t)blockIdx.x * R::RPB; first < p.rows; first += step) {
    const int64_t row = first + threadIdx.x / R::LPR, at = row * p.width;
    const bool keep = row < p.rows;
    float n[R::E], g[R::E], d[R::E];
    R::take(n, rx);
    R::take(d, rd);
    if (p.gate) R::take(g, rg);
    ask(row + step);
    const float rstd = normalize<R>(n, p.width, p.center, p.eps, l, sh, turn);
    if (p.gate) {
#pragma unroll
      for (int j = 0; j < R::E; ++j) {
        const float sig = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g[j]));
        const float act = g[j] * sig;
        g[j] = d[j] * n[j] * w[j] * (sig + act * (1.f - sig));
        d[j] *= act;
      }
      if (keep) R::store(reinterpret_cast<T*>(p.dgate) + at, g, p.width, l);
    }
#pragma unroll
    for (int j = 0; j < R::E; ++j) {
      acc[j] += d[j] * n[j];
      d[j] *= w[j];
    }
    normalize_grad<R>(d, n, rstd, p.width, p.center, sh, turn);
    if (keep) R::store(reinterpret_cast<T*>(p.dx) + at, d, p.width, l);
  }
  if (p.dweight) put_sums<R>(acc, p.partial + (int64_t)blockIdx.x * p.width, p.width, lds);
}

template <typename T, typename R>
__global__ __launch_bounds__(R::THREADS) void residual_norm_bwd_kernel(NormParams p) {
  __shared__ float sh[64];
  __shared__ float lds[R::RPB == 1 ? 1 : R::THREADS * R::E];
  int turn = 0;
  const int l = threadIdx.x % R::LPR;
  float w[R::E], post[R::E], scale[R::E], aw[R::E], ap[R::E], as[R::E];
  R::load(w, p.weight, p.width, l);
  if (p.post) R::load(post, p.post, p.width, l);
  if (p.scale) R::load(scale, p.scale, p.width, l);
#pragma unroll
  for (int j = 0; j < R::E; ++j) {
    if (!p.scale) scale[j] = 1.f;
    aw[j] = ap[j] = as[j] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * R::RPB;
  typename R::Raw rx, ry, rd, rr;
  auto ask = [&](int64_t row) {
    const int64_t at = row * p.width;
    const bool keep = row < p.rows;
    R::ask(rx, reinterpret_cast<const T*>(p.x) + at, p.width, l, keep);
    R::ask(ry, reinterpret_cast<const T*>(p.y) + at, p.width, l, keep);
    R::ask(rd, reinterpret_cast<const T*>(p.dout) + at, p.width, l, keep);
    if (p.dresidual) R::ask(rr, reinterpret_cast<const T*>(p.dresidual) + at, p.width, l, keep);
  };
  ask((int64_t)blockIdx.x * R::RPB + threadIdx.x / R::LPR);
  for (int64_t first = (int64_t)blockIdx.x * R::RPB; first < p.rows; first += step) {
    const int64_t row = first + threadIdx.x / R::LPR, at = row * p.width;
    const bool keep = row < p.rows;
    float h[R::E], y[R::E], g[R::E], r[R::E];
    R::take(h, rx);
    R::take(y, ry);
    R::take(g, rd);
    if (p.dresidual) R::take(r, rr);
    ask(row + step);
    float rstd_y = 0.f;
    if (p.post) rstd_y = normalize<R>(y, p.width, p.center, p.eps, l, sh, turn);
#pragma unroll
    for (int j = 0; j < R::E; ++j) h[j] = p.skip * h[j] + scale[j] * (p.post ? y[j] * post[j] : y[j]);
    const float rh = normalize<R>(h, p.width, p.center, p.eps, l, sh, turn);
#pragma unroll
    for (int j = 0; j < R::E; ++j) {
      aw[j] += g[j] * h[j];
      g[j] *= w[j];
    }
    normalize_grad<R>(g, h, rh, p.width, p.center, sh, turn);
    if (p.dresidual) {
#pragma unroll
      for (int j = 0; j < R::E; ++j) g[j] += r[j];
    }
#pragma unroll
    for (int j = 0; j < R::E; ++j) h[j] = p.skip * g[j];
    if (keep) R::store(reinterpret_cast<T*>(p.dx) + at, h, p.width, l);
#pragma unroll
    for (int j = 0; j < R::E; ++j) {
      as[j] += g[j] * (p.post ? y[j] * post[j] : y[j]);
      g[j] *= scale[j];
    }
    if (p.post) {
#pragma unroll
      for (int j = 0; j < R::E; ++j) {
        ap[j] += g[j] * y[j];
        g[j] *= post[j];
      }
      normalize_grad<R>(g, y, rstd_y, p.width, p.center, sh, turn);
    }
    if (keep) R::store(reinterpret_cast<T*>(p.dy) + at, g, p.width, l);
  }
  const int64_t at = (int64_t)blockIdx.x * p.width, sums = (int64_t)gridDim.x * p.width;
  put_sums<R>(aw, p.partial + at, p.width, lds);
  if (p.post) put_sums<R>(ap, p.partial + sums + at, p.width, lds);
  if (p.scale) put_sums<R>(as, p.partial + 2 * sums + at, p.width, lds);
}

// out[c] = sum over blocks of partial[block][c], 64 columns a workgroup, 16
// strands of blocks added in order. blockIdx.y: which of the sums.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* partial, int blocks, int width, float* o0,
                                                          float* o1, float* o2) {
  __shared__ float s[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), strand = threadIdx.x >> 6;
  const float* at = partial + (int64_t)blockIdx.y * blocks * width + c;
  float x = 0.f;
  if (c < width)
#pragma unroll 8
    for (int b = strand; b < blocks; b += 16) x += at[(int64_t)b * width];
  s[strand][threadIdx.x & 63] = x;
  __syncthreads();
  if (strand == 0 && c < width) {
    x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += s[i][threadIdx.x];
    out[c] = x;
  }
}

// Enough workgroups to fill the chip (2048 lanes a CU), and rows enough for
// each that their sums' traffic stays small beside the rows'.
int norm_bwd_blocks(int64_t rows, int width) {
  int threads = 256, rpb = 1;
  if (width > 8192) threads = 1024;
  else if (width > 2048) threads = 512;
  else for (rpb = 32; rpb > 1 && 2048 / rpb < width;) rpb /= 2;
  const int64_t most = 256 * (1024 / threads), need = (rows + rpb - 1) / rpb;
  return (int)(need < 1 ? 1 : need < most ? need : most);  // without rows: sums of zero
}

template <typename T>
static hipError_t launch_bwd(const NormParams& p, bool residual, hipStream_t stream) {
  const int blocks = norm_bwd_blocks(p.rows, p.width);
  const hipError_t e = with_rows<T, true>(p.width, p.width % 8 == 0, [&](auto r) {
    using R = decltype(r);
    if (residual)
      hipLaunchKernelGGL((residual_norm_bwd_kernel<T, R>), dim3(blocks), dim3(R::THREADS), 0, stream, p);
    else
      hipLaunchKernelGGL((head_norm_bwd_kernel<T, R>), dim3(blocks), dim3(R::THREADS), 0, stream, p);
    return hipGetLastError();
  });
  if (e != hipSuccess || !(p.dweight || p.dpost || p.dscale)) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((p.width + 63) / 64, residual ? 3 : 1), dim3(1024), 0, stream, p.partial,
                     blocks, p.width, p.dweight, p.dpost, p.dscale);
  return hipGetLastError();
}

hipError_t launch_head_norm_bwd(const NormParams& p, int dtype, hipStream_t stream) {
  return dtype == 1 ? launch_bwd<bf16>(p, false, stream) : launch_bwd<float>(p, false, stream);
}
hipError_t launch_residual_norm_bwd(const NormParams& p, int dtype, hipStream_t stream) {
  return dtype == 1 ? launch_bwd<bf16>(p, true, stream) : launch_bwd<float>(p, true, stream);
}

}  // namespace ret
