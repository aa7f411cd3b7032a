// Gated linear recurrence, gradients. With g_t = dout_t + a_(t+1) g_(t+1) and s_i,
// s_d the sigmoids of gate and decay:
//     dx = g m s_i,   dgate = g m x s_i (1 - s_i),
//     dla = a g h_(t-1) - (a^2 / m) g s_i x   (the second term with normalize)
//     ddecay = dla, or -rate s_d (1 - s_d) dla;   drate = -sum of s_d dla
//     d state_in = a_0 g_0
// Laid out as the forward, over tiles of 128 tokens (a segment holds twice its values
// a token): the tile's states are formed again from the one kept before it, and the
// gradient of the state behind it comes from the tile after it, as a word in memory.
// Tiles start from the last. A tile's share of drate goes to a row of sums that a
// second launch adds up in a fixed order. The gradients' stores bypass the caches, which
// leaves the inputs there. Past them and through them, forward and gradients one after the
// other over changing inputs; with inputs in memory and dout just written, the call and
// the convolution's gradients after it; these and products that read all gradients: 4 x 2048 x
// 2560 115 / 115 / 253 us and 120 / 114 / 251, 2 x 8192 x 4096 295 / 290 / 606 and 305 / 300 /
// 618, 8 x 2048 x 1024 98 / 98 / 204 and 105 / 97 / 203. Not where rows end inside a line of 128
// bytes, whose parts two workgroups write: 4 x 8192 x 4100 609 us a call through the caches and
// 784 past them, 2 x 8192 x 4095 284 and 346, 2 x 4096 x 6000 189 and 207.
// Measured in bf16 with both gates, kernel alone: 4 x 2048 x 2560 70 us (4.2 TB/s), 4 x 8192 x
// 4100 600 us; calls of 2 x 8192 x 4096 191 us, 1 x 16384 x 8192 362 us (5.2 TB/s), 1 x 32768 x
// 1024 172 us (the chain of 256 tiles), 1 x 131072 x 2560 1170 us (4.0 TB/s); fp32, kernel
// alone, 2 x 8192 x 2048 195 us (4.8 TB/s).
// Bound by memory and arithmetic together: the SIMDs compute in 59 % of
// their cycles (71 vector instructions for 64 elements), waves wait in 37 % of theirs for
// memory. 128 registers a lane, two workgroups a CU: one of each fetches while the other computes.
#include "norms.hpp"
#include "scan_common.hpp"

// The variants of a kernel give the same bits: fused multiply-adds only where they are written.
#pragma clang fp contract(off)

namespace ret {

constexpr int kSegment = 8;  // tokens; 16 segments a tile

template <typename T, bool GATES, bool IGATE, bool NORM, int V>
__global__ __launch_bounds__(kScanBwdTile * 4, 4) void scan_bwd_kernel(ScanParams p) {
  using D = std::conditional_t<GATES, T, float>;
  constexpr int LW = kScanChannels / V, PARTS = 2 / V, L = kSegment * PARTS, SEGS = kScanBwdTile / kSegment;
  __shared__ float s_a[SEGS][kScanChannels], s_u[SEGS][kScanChannels], s_p[SEGS][kScanChannels],
      s_r[SEGS][kScanChannels], s_pr[SEGS][kScanChannels], s_back[kScanChannels];
  // exponents of products (s_a, s_p) that are no normal number; s_odd: whether a wave has some
  __shared__ int s_e[SEGS][kScanChannels], s_pe[SEGS][kScanChannels], s_odd[SEGS / 2];
  clear_errors(p);
  const Place at = place_of<true>(p, kScanBwdTile);
  if (!at.any) return;
  int tok0, len;
  span_of(p, at.b, tok0, len);
  const int from = at.i * kScanBwdTile;
  const int lane = threadIdx.x & 63, wave = uniform_i(threadIdx.x >> 6);
  const int c0 = at.group * kScanChannels, ch = c0 + lane;
  if (from >= len && !(at.i == 0 && len == 0)) {
    if (GATES && wave == 0 && ch < p.width) p.partial[at.tile * p.width + ch] = 0.f;
    return;
  }
  const int seg = wave * 2 + lane / LW, cl = lane % LW * V;  // the lane's first segment
  const int c = min(c0 + cl, p.width - V);
  const bool inside = c0 + cl < p.width;
  T* dx = reinterpret_cast<T*>(p.dx);
  D* ddecay = reinterpret_cast<D*>(p.ddecay);
  T* dgate = reinterpret_cast<T*>(p.dgate);
  if (p.cu && at.i == 0) {
    // rows before the first sequence and behind the last have gradient 0
    auto clear = [&](int t0, int t1) {
      const float zero[V] = {};
      // a row for each wave, with pairs of channels for each half of one
      for (int64_t t = t0 + (V == 1 ? wave : seg); t < t1 && inside; t += V == 1 ? SEGS / 2 : SEGS) {
        lane_store<T, V>(dx + t * p.width, c, zero);
        lane_store<D, V>(ddecay + t * p.width, c, zero);
        if constexpr (IGATE) lane_store<T, V>(dgate + t * p.width, c, zero);
      }
    };
    if (at.b == 0) clear(0, tok0);
    if (at.b == p.batch - 1) clear(tok0 + len, p.total);
  }
  const int left = len - from, n = left - seg * kSegment;  // tokens from the tile's, the lane's start on
  const int there = min(left, kScanBwdTile);
  const int64_t row = (int64_t)tok0 + from;
  lane_raw<T, V> rx[L], ro[L];
  // sd, si: the sigmoids; rest: 1 - a^2; hist: inputs, then the state before each token
  float a[L][V], sd[GATES ? L : 1][V], si[IGATE ? L : 1][V], rest[NORM && !GATES ? L : 1][V], hist[L][V];
  float A[PARTS][V], U[PARTS][V], R[PARTS][V], rate[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    rate[e] = GATES ? p.rate[c + e] : 0.f;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      A[k][e] = 1.f;
      U[k][e] = R[k][e] = 0.f;
    }
  }

  auto fold = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.x_stride;
    const D* decay = reinterpret_cast<const D*>(p.decay) + row * p.decay_stride;
    const T* gate = reinterpret_cast<const T*>(p.gate) + (IGATE ? row * p.gate_stride : 0);
    const T* dout = reinterpret_cast<const T*>(p.dout) + row * p.width;
    lane_raw<T, V> rg[IGATE ? L : 1];
    lane_raw<D, V> rd[L];
    const Rows<T, V> xs(x, p.x_stride, there, p.width, seg * kSegment, c);
    const Rows<D, V> ds(decay, p.decay_stride, there, p.width, seg * kSegment, c);
    const Rows<T, V> gs(gate, p.gate_stride, there, p.width, seg * kSegment, c);
    const Rows<T, V> os(dout, p.width, there, p.width, seg * kSegment, c);
#pragma unroll
    for (int j = 0; j < L; ++j) {
      rx[j] = FULL ? xs.load(j) : xs.load_if(j);
      rd[j] = FULL ? ds.load(j) : ds.load_if(j);
      if constexpr (IGATE) rg[j] = FULL ? gs.load(j) : gs.load_if(j);
      ro[j] = FULL ? os.load(j) : os.load_if(j);
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
      float d[V], g[V];
      Lane<D, V>::get(rd[j], d);
      Lane<T, V>::get(rx[j], hist[j]);
      if constexpr (IGATE) Lane<T, V>::get(rg[j], g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float la = d[e], q;
        if constexpr (GATES) {
          sd[j][e] = sigmoid_of(d[e], T());
          la = -rate[e] * sd[j][e];
        }
        factor<T>(la, a[j][e], q);
        if constexpr (IGATE) {
          si[j][e] = sigmoid_of(g[e], T());
          hist[j][e] *= si[j][e];
        }
        if constexpr (NORM) {
          if constexpr (!GATES) rest[j][e] = q;  // (formed again from s_d: 16 registers less)
          hist[j][e] *= __builtin_amdgcn_sqrtf(q);
        }
        if (!FULL && j >= n) {  // behind the end
          a[j][e] = 1.f;
          hist[j][e] = 0.f;
        }
        float &A1 = A[j / kSegment][e], &U1 = U[j / kSegment][e];
        U1 = fmaf(a[j][e], U1, hist[j][e]);
        A1 *= a[j][e];
      }
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      float d[V];
      Lane<T, V>::get(ro[j], d);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (FULL || j < n) R[j / kSegment][e] = a[j][e] * (R[j / kSegment][e] + d[e]);
    }
  };
  const bool full = left >= kScanBwdTile;
  if (full)
    fold(std::true_type());
  else if (wave * 2 * kSegment < left)
    fold(std::false_type());
  // a product that is no normal number: exact, and sums that forget what stood before them
  bool odd = false;
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) odd |= !is_normal(A[k][e]);
  odd = __any(odd);
  if (odd) {
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float& U1 = U[j / kSegment][e];
        U1 = j % kSegment ? step_or_forget(a[j][e], U1, hist[j][e]) : hist[j][e];
      }
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      float d[V];
      Lane<T, V>::get(ro[j], d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float& R1 = R[j / kSegment][e];
        if ((j + 1) % kSegment == 0) R1 = 0.f;
        if (j < n) R1 = a[j][e] == 0.f ? 0.f : a[j][e] * (R1 + d[e]);
      }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (!is_normal(A[k][e])) {
          Growing t;
          bool none = false;
#pragma unroll
          for (int j = 0; j < kSegment; ++j) {
            none |= a[k * kSegment + j][e] == 0.f;
            t.by(a[k * kSegment + j][e]);
          }
          A[k][e] = none ? 0.f : -t.m;
          s_e[seg + k][cl + e] = t.e;
        }
  }
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s_a[seg + k][cl + e] = A[k][e];
      s_u[seg + k][cl + e] = U[k][e];
      s_r[seg + k][cl + e] = R[k][e];
    }
  if (lane == 0) s_odd[wave] = odd;
  __syncthreads();
  const bool mine = ch < p.width, any_odd = __any(s_odd[lane % (SEGS / 2)]);
  if (wave == 0) {
    // gradients from behind
    const bool last = left <= kScanBwdTile;
    const int64_t held = (int64_t)at.b * p.width + ch;
    float ta = 1.f, tr = 0.f, low = 1.f;
#pragma unroll
    for (int s = SEGS - 1; s >= 0; --s) {
      const float sa = s_a[s][lane], sr = s_r[s][lane];
      s_p[s][lane] = ta;
      s_pr[s][lane] = tr;
      tr = fmaf(sa, tr, sr);
      ta *= sa;
      low = fminf(low, ta);
    }
    bool far = !is_normal(ta) || !is_normal(low);
    if (any_odd)
      for (int s = 0; s < SEGS; ++s) far |= !is_normal(s_a[s][lane]);
    const bool any_far = __any(far);
    Product total = {ta, 0};
    if (far) {
      Growing t;
      if (any_odd) {
        tr = 0.f;
#pragma unroll 4
        for (int s = SEGS - 1; s >= 0; --s) {
          const Product one = {s_a[s][lane], s_e[s][lane]};
          s_p[s][lane] = -t.m;
          s_pe[s][lane] = t.e;
          s_pr[s][lane] = tr;
          tr = step_over(one, tr, s_r[s][lane]);
          t.by(one);
        }
      } else {  // (the sums as they are: every segment's factor is a normal number)
#pragma unroll
        for (int s = SEGS - 1; s >= 0; --s) {
          s_p[s][lane] = -t.m;
          s_pe[s][lane] = t.e;
          t.by(s_a[s][lane]);
        }
      }
      total = t.product();
    }
    float back = 0.f;
    if (!last)
      back = take_over(p.hand + (at.tile + 1) * p.width + ch, mine, p.ctrl);
    else if (p.d_state_out && mine)
      back = p.d_state_out[held];
    s_back[lane] = back;
    back = any_far ? step_over(total, back, tr) : fmaf(ta, back, tr);
    if (mine) {
      if (at.i > 0)
        hand_on(p.hand + at.tile * p.width + ch, back);
      else if (p.d_state_in)
        p.d_state_in[held] = back;
    }
  } else if (wave == 1) {
    // states from before
    float h = 0.f;
    if (mine && len > 0) h = p.kept[(kept_row(p, at.b, tok0) + at.i) * p.width + ch];
    if (any_odd) {
#pragma unroll 1
      for (int s = 0; s < SEGS; ++s) {
        const float su = s_u[s][lane];
        s_u[s][lane] = h;
        h = step_over({s_a[s][lane], s_e[s][lane]}, h, su);
      }
    } else {
      float before[SEGS];
#pragma unroll
      for (int s = 0; s < SEGS; ++s) {
        before[s] = h;
        h = fmaf(s_a[s][lane], h, s_u[s][lane]);
      }
#pragma unroll
      for (int s = 0; s < SEGS; ++s) s_u[s][lane] = before[s];
    }
  }
  __syncthreads();
  float sum[PARTS][V] = {};
  auto run = [&](auto whole, auto forget, auto stream) {
    constexpr bool FULL = decltype(whole)::value, FORGET = decltype(forget)::value;
    constexpr int POLICY = decltype(stream)::value ? kStreamed : 0;
    float h[V], g[V];  // g: what reaches the token's state from behind
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (j % kSegment == 0) h[e] = s_u[seg + j / kSegment][cl + e];
        const float u = hist[j][e];
        hist[j][e] = h[e];
        h[e] = FORGET ? step_or_forget(a[j][e], h[e], u) : fmaf(a[j][e], h[e], u);
      }
    }
    const Rows<T, V> to_x(dx + row * p.width, p.width, there, p.width, seg * kSegment, c, inside);
    const Rows<D, V> to_decay(ddecay + row * p.width, p.width, there, p.width, seg * kSegment, c, inside);
    const Rows<T, V> to_gate(dgate + (IGATE ? row * p.width : 0), p.width, there, p.width, seg * kSegment, c,
                             inside);
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
      float xs[V], d[V], o1[V], o2[V], o3[V];
      if ((j + 1) % kSegment == 0) {
        const int k = seg + j / kSegment;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          g[e] = step_over(s_p[k][cl + e], &s_pe[k][cl + e], s_back[cl + e], s_pr[k][cl + e]);
        }
      }
      Lane<T, V>::get(rx[j], xs);
      Lane<T, V>::get(ro[j], d);
      if (FULL || j < n) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          g[e] += d[e];
          const float s = IGATE ? si[j][e] : 1.f, av = a[j][e];
          // a token that forgets lets no gradient through, whatever reaches it
          const bool none = FORGET && av == 0.f;
          const float ag = none ? 0.f : av * g[e];
          float dla = none ? 0.f : ag * hist[j][e], m = 1.f, r = 0.f;
          if constexpr (NORM) {
            // a / m; 0 where the decay is 0, the limit towards which ddecay goes
            float q;
            if constexpr (GATES)
              q = left_of<T>(-rate[e] * sd[j][e], av);
            else
              q = rest[j][e];
            // (below the normal numbers too: the hardware's root takes those for 0)
            const float inv = q >= 0x1p-126f ? __builtin_amdgcn_rsqf(q) : 0.f;
            m = q * inv;
            r = av * inv;
          }
          o1[e] = g[e] * m * s;
          const float to_gated = o1[e] * xs[e];  // g m s_i x
          if constexpr (NORM) dla = none ? 0.f : fmaf(-r * r, to_gated, dla);
          if constexpr (IGATE) o3[e] = fmaf(-s, to_gated, to_gated);
          if constexpr (GATES) {
            const float t = sd[j][e] * dla;
            sum[j / kSegment][e] -= t;
            o2[e] = fmaf(rate[e], sd[j][e], -rate[e]) * t;
          } else {
            o2[e] = dla;
          }
          g[e] = ag;
        }
        to_x.template store<POLICY>(j, o1);
        to_decay.template store<POLICY>(j, o2);
        if constexpr (IGATE) to_gate.template store<POLICY>(j, o3);
      }
    }
  };
  if (wave * 2 * kSegment < left) {
    // rows of whole lines, or parts of a line have to meet in the L2
    const bool lines = (uint32_t)p.width * (uint32_t)sizeof(T) % 128 == 0;
    if (odd)
      run(std::false_type(), std::true_type(), std::false_type());
    else if (full && lines)
      run(std::true_type(), std::false_type(), std::true_type());
    else if (full)
      run(std::true_type(), std::false_type(), std::false_type());
    else
      run(std::false_type(), std::false_type(), std::false_type());
  }
  if constexpr (GATES) {
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s_a[seg + k][cl + e] = sum[k][e];
    __syncthreads();
    if (wave == 0 && mine) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < SEGS; ++k) s += s_a[k][lane];
      p.partial[at.tile * p.width + ch] = s;
    }
  }
}

template <typename T, bool GATES, bool IGATE, bool NORM, int V>
static hipError_t launch_bwd(const ScanParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((scan_bwd_kernel<T, GATES, IGATE, NORM, V>), dim3(scan_grid(p)), dim3(kScanBwdTile * 4), 0,
                     stream, p);
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
  hipError_t e = launch_scan_prep(p, stream);
  if (e != hipSuccess) return e;
  e = dtype != 1     ? launch_bwd_v<float, 1>(p, stream)
      : in_pairs(p) ? launch_bwd_v<bf16, 2>(p, stream)
                    : launch_bwd_v<bf16, 1>(p, stream);
  if (e != hipSuccess || !p.rate) return e;
  return launch_column_sum(p.partial, p.tiles, p.width, p.drate, stream);
}

}  // namespace ret
