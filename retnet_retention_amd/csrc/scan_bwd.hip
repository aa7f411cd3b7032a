// Gated linear recurrence, gradients. With g_t = dout_t + a_(t+1) g_(t+1) and s_i,
// s_d the sigmoids of gate and decay:
//     dx = g m s_i,   dgate = g m x s_i (1 - s_i),
//     dla = a g h_(t-1) - (a^2 / m) g s_i x   (the second term with normalize)
//     ddecay = dla, or -rate s_d (1 - s_d) dla;   drate = -sum of s_d dla
//     d state_in = a_0 g_0
// A workgroup walks a sequence's tiles from the last to the first for the 64 V
// channels of its lanes. A tile's states are formed again from the state kept before
// it; each wave folds its tokens both ways, and what the waves hand each other goes
// through LDS once a tile.
#include "norms.hpp"
#include "scan_common.hpp"

namespace ret {

template <typename T, bool GATES, bool IGATE, bool NORM, int V, int L, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void scan_bwd_kernel(ScanParams p) {
  using D = std::conditional_t<GATES, T, float>;
  static_assert(L * WAVES == kScanTile, "");
  __shared__ float s_a[2][WAVES][64 * V], s_u[2][WAVES][64 * V], s_r[2][WAVES][64 * V];
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int groups = (p.width + 64 * V - 1) / (64 * V);
  const int b = blockIdx.x / groups, at = (blockIdx.x % groups * 64 + lane) * V;
  const bool inside = at < p.width;
  const int c = min(at, p.width - V);
  int tok0, len;
  span_of(p, b, tok0, len);
  float rate[V], back[V], sum[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    rate[e] = GATES ? p.rate[c + e] : 0.f;
    back[e] = p.d_state_out ? p.d_state_out[(int64_t)b * p.width + c + e] : 0.f;
    sum[e] = 0.f;
  }
  const int64_t first_tile = p.cu ? tok0 / kScanTile + b : (int64_t)b * ((p.seqlen + kScanTile - 1) / kScanTile);
  const T* x = reinterpret_cast<const T*>(p.x) + tok0 * p.x_stride;
  const D* decay = reinterpret_cast<const D*>(p.decay) + tok0 * p.decay_stride;
  const T* gate = reinterpret_cast<const T*>(p.gate) + (IGATE ? tok0 * p.gate_stride : 0);
  const int64_t row0 = (int64_t)tok0 * p.width;
  const T* dout = reinterpret_cast<const T*>(p.dout) + row0;
  T* dx = reinterpret_cast<T*>(p.dx) + row0;
  D* ddecay = reinterpret_cast<D*>(p.ddecay) + row0;
  T* dgate = reinterpret_cast<T*>(p.dgate) + (IGATE ? row0 : 0);
  // rows before the first sequence and behind the last have gradient 0
  auto clear = [&](int from, int to) {
    const float zero[V] = {};
    for (int t = from + wave; t < to && inside; t += WAVES) {
      const int64_t r = ((int64_t)t - tok0) * p.width;
      lane_store<T, V>(dx + r, c, zero);
      lane_store<D, V>(ddecay + r, c, zero);
      if constexpr (IGATE) lane_store<T, V>(dgate + r, c, zero);
    }
  };
  if (p.cu && b == 0) clear(0, tok0);
  if (p.cu && b == p.batch - 1) clear(tok0 + len, p.total);
  int turn = 0;
  for (int base = (len - 1) / kScanTile * kScanTile; len > 0 && base >= 0; base -= kScanTile, turn ^= 1) {
    const int t0 = base + wave * L, n = min(max(len - t0, 0), L);
    lane_raw<T, V> rx[L], rg[IGATE ? L : 1], ro[L];
    lane_raw<D, V> rd[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int t = min(t0 + j, len - 1);
      rx[j] = lane_load<T, V>(x + t * p.x_stride, c);
      rd[j] = lane_load<D, V>(decay + t * p.decay_stride, c);
      if constexpr (IGATE) rg[j] = lane_load<T, V>(gate + t * p.gate_stride, c);
      ro[j] = lane_load<T, V>(dout + (int64_t)t * p.width, c);
    }
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = p.kept[(first_tile + base / kScanTile) * p.width + c + e];
    // sd, si: the sigmoids; hist: u, then the state before the token
    float a[L][V], sd[GATES ? L : 1][V], si[IGATE ? L : 1][V], left[NORM ? L : 1][V], hist[L][V];
    float A[V], U[V], R[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      A[e] = 1.f;
      U[e] = R[e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float d[V], g[V];
      Lane<D, V>::get(rd[j], d);
      Lane<T, V>::get(rx[j], hist[j]);
      if constexpr (IGATE) Lane<T, V>::get(rg[j], g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float la = d[e], lf;
        if constexpr (GATES) {
          sd[j][e] = sigmoid_of(d[e], T());
          la = -rate[e] * sd[j][e];
        }
        factor<T>(la, a[j][e], lf);
        if constexpr (IGATE) {
          si[j][e] = sigmoid_of(g[e], T());
          hist[j][e] *= si[j][e];
        }
        if constexpr (NORM) {
          left[j][e] = lf;
          hist[j][e] *= __builtin_amdgcn_sqrtf(lf);
        }
        if (j >= n) {  // behind the end
          a[j][e] = 1.f;
          hist[j][e] = 0.f;
        }
        U[e] = step_or_forget(a[j][e], U[e], hist[j][e]);
        A[e] *= a[j][e];
      }
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      float d[V];
      Lane<T, V>::get(ro[j], d);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (j < n) R[e] = a[j][e] == 0.f ? 0.f : a[j][e] * (R[e] + d[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s_a[turn][wave][lane * V + e] = A[e];
      s_u[turn][wave][lane * V + e] = U[e];
      s_r[turn][wave][lane * V + e] = R[e];
    }
    __syncthreads();
    float g[V];
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      if (w < wave) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = step_or_forget(s_a[turn][w][lane * V + e], h[e], s_u[turn][w][lane * V + e]);
      }
#pragma unroll
    for (int w = WAVES - 1; w >= 0; --w) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (w == wave) g[e] = back[e];
        back[e] = step_or_forget(s_a[turn][w][lane * V + e], back[e], s_r[turn][w][lane * V + e]);
      }
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u = hist[j][e];
        hist[j][e] = h[e];
        h[e] = step_or_forget(a[j][e], h[e], u);
      }
    }
    // g: what reaches the token's state from behind
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      float xs[V], d[V], o1[V], o2[V], o3[V];
      Lane<T, V>::get(rx[j], xs);
      Lane<T, V>::get(ro[j], d);
      if (j < n) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          g[e] += d[e];
          const float s = IGATE ? si[j][e] : 1.f, av = a[j][e];
          // a token that forgets lets no gradient through, whatever reaches it
          const float ag = av == 0.f ? 0.f : av * g[e];
          float dla = av == 0.f ? 0.f : ag * hist[j][e], m = 1.f;
          if constexpr (NORM) {
            // a^2 / m; 0 where the decay is 0, the limit towards which ddecay goes
            const float inv = left[j][e] > 0.f ? __builtin_amdgcn_rsqf(left[j][e]) : 0.f;
            m = left[j][e] * inv;
            dla -= ag * av * inv * s * xs[e];
          }
          const float gm = g[e] * m;
          o1[e] = gm * s;
          if constexpr (IGATE) o3[e] = o1[e] * xs[e] * (1.f - s);
          if constexpr (GATES) {
            const float t = sd[j][e] * dla;
            sum[e] -= t;
            o2[e] = -rate[e] * (1.f - sd[j][e]) * t;
          } else {
            o2[e] = dla;
          }
          g[e] = ag;
        }
        if (inside) {
          lane_store<T, V>(dx + (int64_t)(t0 + j) * p.width, c, o1);
          lane_store<D, V>(ddecay + (int64_t)(t0 + j) * p.width, c, o2);
          if constexpr (IGATE) lane_store<T, V>(dgate + (int64_t)(t0 + j) * p.width, c, o3);
        }
      }
    }
  }
  if (p.d_state_in && wave == 0 && inside) {
#pragma unroll
    for (int e = 0; e < V; ++e) p.d_state_in[(int64_t)b * p.width + c + e] = back[e];
  }
  if constexpr (GATES) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) s_a[0][wave][lane * V + e] = sum[e];
    __syncthreads();
    if (wave == 0 && inside) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += s_a[0][w][lane * V + e];
        p.partial[(int64_t)b * p.width + c + e] = s;
      }
    }
  }
}

template <typename T, bool GATES, bool IGATE, bool NORM, int V>
static hipError_t launch_bwd(const ScanParams& p, hipStream_t stream) {
  constexpr int L = 8, WAVES = kScanTile / L;
  const int64_t groups = (p.width + 64 * V - 1) / (64 * V);
  hipLaunchKernelGGL((scan_bwd_kernel<T, GATES, IGATE, NORM, V, L, WAVES>), dim3((unsigned)(groups * p.batch)),
                     dim3(WAVES * 64), 0, stream, p);
  return hipGetLastError();
}
template <typename T, int V>
static hipError_t launch_bwd_v(const ScanParams& p, hipStream_t s) {
  const int which = (p.rate ? 4 : 0) + (p.gate ? 2 : 0) + (p.normalize ? 1 : 0);
  switch (which) {
    case 0: return launch_bwd<T, false, false, false, V>(p, s);
    case 1: return launch_bwd<T, false, false, true, V>(p, s);
    case 2: return launch_bwd<T, false, true, false, V>(p, s);
    case 3: return launch_bwd<T, false, true, true, V>(p, s);
    case 4: return launch_bwd<T, true, false, false, V>(p, s);
    case 5: return launch_bwd<T, true, false, true, V>(p, s);
    case 6: return launch_bwd<T, true, true, false, V>(p, s);
    default: return launch_bwd<T, true, true, true, V>(p, s);
  }
}
hipError_t launch_scan_bwd(const ScanParams& p, int dtype, hipStream_t stream) {
  if (p.cu) {
    const hipError_t e = launch_check_bounds(p.cu, p.batch, p.total, p.ctrl, stream);
    if (e != hipSuccess) return e;
  }
  hipError_t e = dtype != 1 ? launch_bwd_v<float, 1>(p, stream)
                 : in_pairs(p) ? launch_bwd_v<bf16, 2>(p, stream)
                            : launch_bwd_v<bf16, 1>(p, stream);
  if (e != hipSuccess || !p.rate) return e;
  return launch_column_sum(p.partial, p.batch, p.width, p.drate, stream);
}

}  // namespace ret
