// C-ABI host layer of the gated delta rule: argument validation, workspace
// carving and launches on the caller's stream.
#include <cmath>

#include "delta.hpp"
#include "host_checks.hpp"

namespace {

using namespace ret_host;
using ret::DeltaLayout;
using ret::DeltaParams;

constexpr int kMaxHeads = 128;

ret_status_t check_delta(const ret_delta_desc_t* d, bool packed, int64_t total) {
  if (!d) return RET_ERR_NULL;
  if (d->batch < 1 || d->seqlen < 1 || d->k_heads < 1 || d->v_heads < 1 || d->v_heads > kMaxHeads ||
      d->v_heads % d->k_heads != 0)
    return RET_ERR_SHAPE;
  // rows are numbered with 32 bits, and so are the threads of a launch: 512 for
  // each of a head's (up to 8) slices, or for each block of 64 tokens
  const int64_t tokens = (int64_t)d->batch * d->seqlen;
  const int64_t blocks = (int64_t)d->batch * ((d->seqlen + (int64_t)ret::kDeltaBlock - 1) / ret::kDeltaBlock);
  if (tokens > INT32_MAX || (int64_t)d->batch * d->v_heads >= 1 << 20 || blocks >= 1 << 23) return RET_ERR_SHAPE;
  if (packed && (total < 0 || total > tokens)) return RET_ERR_SHAPE;
  if (d->dtype != RET_F32 && d->dtype != RET_BF16) return RET_ERR_UNSUPPORTED;
  if (d->dk != d->dv || (d->dk != 64 && d->dk != 128 && d->dk != 256)) return RET_ERR_UNSUPPORTED;
  if (!std::isfinite(d->scale)) return RET_ERR_ARG;
  return RET_OK;
}

struct Sizes {
  size_t tokens, qk, v, gate, state;
};
Sizes sizes_of(const ret_delta_desc_t* d, bool packed, int64_t total) {
  Sizes s;
  s.tokens = packed ? (size_t)total : (size_t)d->batch * d->seqlen;
  s.qk = s.tokens * d->k_heads * d->dk * elem_size(d->dtype);
  s.v = s.tokens * d->v_heads * d->dv * elem_size(d->dtype);
  s.gate = s.tokens * d->v_heads * sizeof(float);
  s.state = (size_t)d->batch * d->v_heads * d->dk * d->dv * sizeof(float);
  return s;
}

DeltaLayout layout_of(const ret_delta_desc_t* d, bool packed, int64_t total) {
  return ret::delta_layout(d->batch, d->seqlen, d->dtype, packed, (int)total);
}

// Takes 256-byte aligned parts of a workspace in turn; with no workspace it
// only counts.
struct Carve {
  char* base;
  size_t used = 0;
  template <typename P>
  void part(P*& p, size_t bytes) {
    p = base ? reinterpret_cast<P*>(base + used) : nullptr;
    used += align_up(bytes);
  }
};

size_t key_bytes(const DeltaLayout& l, const ret_delta_desc_t* d) {
  return l.blocks * d->k_heads * ret::kDeltaBlock * d->dk * elem_size(d->dtype);
}

// control block | T | decay vectors | keys in the lanes' order
void carve_shared(Carve& c, DeltaParams& p, const DeltaLayout& l, const ret_delta_desc_t* d, int planes) {
  const size_t n = l.blocks * d->v_heads;
  c.part(p.ctrl, 2 * sizeof(int32_t));
  c.part(p.t, n * planes * l.mat_plane);
  c.part(p.vec, n * 4 * ret::kDeltaBlock * sizeof(float));
  c.part(p.kf, key_bytes(l, d));
  c.part(p.kc, key_bytes(l, d));
}

// the shared parts | M | queries
void carve_fwd(Carve& c, DeltaParams& p, const DeltaLayout& l, const ret_delta_desc_t* d) {
  carve_shared(c, p, l, d, l.planes);
  c.part(p.m, l.blocks * d->v_heads * l.planes * l.mat_plane);
  c.part(p.qf, key_bytes(l, d));
}

// the shared parts | queries | q.k and k.k | T^T | P^T | states | gradients of states | V' | rest of dv
void carve_bwd(Carve& c, DeltaParams& p, const DeltaLayout& l, const ret_delta_desc_t* d, const Sizes& s) {
  carve_shared(c, p, l, d, l.mat_planes);
  const size_t n = l.blocks * d->v_heads, state = (size_t)d->dk * d->dv * l.planes * elem_size(d->dtype);
  c.part(p.qc, key_bytes(l, d));
  c.part(p.pairs, l.blocks * d->k_heads * 2 * ret::kDeltaBlock * ret::kDeltaBlock * sizeof(float));
  c.part(p.tt, n * l.mat_planes * l.mat_plane);
  c.part(p.pt, n * l.mat_planes * l.mat_plane);
  c.part(p.snap, n * state);
  c.part(p.dsnap, n * state);
  c.part(p.u, s.v * l.planes);
  c.part(p.dv_rest, s.v * (l.planes - 1));
}

size_t workspace_bytes_of(const ret_delta_desc_t* d, bool packed, int64_t total, bool grad) {
  if (check_delta(d, packed, total) != RET_OK) return 0;
  const DeltaLayout l = layout_of(d, packed, total);
  Carve c{nullptr};
  DeltaParams p = {};
  if (grad)
    carve_bwd(c, p, l, d, sizes_of(d, packed, total));
  else
    carve_fwd(c, p, l, d);
  return c.used;
}

DeltaParams params_of(const ret_delta_desc_t* d, const int32_t* cu, const Sizes& s, const void* q, const void* k,
                      const void* v, const float* log_decay, const float* beta, const float* state_in) {
  DeltaParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.log_decay = log_decay;
  p.beta = beta;
  p.cu = cu;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.k_heads = d->k_heads;
  p.heads = d->v_heads;
  p.total = (int)s.tokens;
  p.blocks_max = (d->seqlen + ret::kDeltaBlock - 1) / ret::kDeltaBlock;
  p.scale = d->scale;
  p.state_in = state_in;
  return p;
}

}  // namespace

extern "C" {

size_t retention_delta_workspace_bytes(const ret_delta_desc_t* desc, int32_t packed, int64_t total_tokens) {
  return workspace_bytes_of(desc, packed != 0, total_tokens, false);
}

ret_status_t retention_delta_fwd(const ret_delta_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                 const void* q, const void* k, const void* v, const float* log_decay,
                                 const float* beta, void* o, const float* state_in, float* state_out, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_delta(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const Sizes s = sizes_of(desc, packed, total_tokens);
  if (s.tokens && (!q || !k || !v || !log_decay || !beta || !o)) return RET_ERR_NULL;
  const size_t need = workspace_bytes_of(desc, packed, total_tokens, false);
  const Arg args[] = {{state_in, s.state, 16, false},
                      {state_out, s.state, 16, true},
                      {q, s.qk, 16, false},
                      {k, s.qk, 16, false},
                      {v, s.v, 16, false},
                      {log_decay, s.gate, 4, false},
                      {beta, s.gate, 4, false},
                      {o, s.v, 16, true},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {workspace, need, 16, true}};
  // every workgroup reads its part of state_in before it writes that part
  if ((st = check_args(args, 9, 0, 1)) != RET_OK) return st;
  if (!workspace || workspace_bytes < need) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, 10, 0, 1)) != RET_OK) return st;
  DeltaParams p = params_of(desc, cu_seqlens, s, q, k, v, log_decay, beta, state_in);
  p.o = o;
  p.state_out = state_out;
  Carve c{static_cast<char*>(workspace)};
  carve_fwd(c, p, layout_of(desc, packed, total_tokens), desc);
  return ret::launch_delta_fwd(p, desc->dk, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

size_t retention_delta_bwd_workspace_bytes(const ret_delta_desc_t* desc, int32_t packed, int64_t total_tokens) {
  return workspace_bytes_of(desc, packed != 0, total_tokens, true);
}

ret_status_t retention_delta_bwd(const ret_delta_desc_t* desc, const int32_t* cu_seqlens, int64_t total_tokens,
                                 const void* q, const void* k, const void* v, const float* log_decay,
                                 const float* beta, const void* dout, const float* state_in, const float* d_state_out,
                                 void* dq, void* dk, void* dv, float* d_log_decay, float* d_beta, float* d_state_in,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  ret_status_t st = check_delta(desc, packed, total_tokens);
  if (st != RET_OK) return st;
  const Sizes s = sizes_of(desc, packed, total_tokens);
  if (s.tokens &&
      (!q || !k || !v || !log_decay || !beta || !dout || !dq || !dk || !dv || !d_log_decay || !d_beta))
    return RET_ERR_NULL;
  if ((state_in == nullptr) != (d_state_in == nullptr)) return RET_ERR_NULL;
  const size_t need = workspace_bytes_of(desc, packed, total_tokens, true);
  const Arg args[] = {{q, s.qk, 16, false},
                      {k, s.qk, 16, false},
                      {v, s.v, 16, false},
                      {log_decay, s.gate, 4, false},
                      {beta, s.gate, 4, false},
                      {dout, s.v, 16, false},
                      {state_in, s.state, 16, false},
                      {d_state_out, s.state, 16, false},
                      {cu_seqlens, ((size_t)desc->batch + 1) * sizeof(int32_t), 4, false},
                      {dq, s.qk, 16, true},
                      {dk, s.qk, 16, true},
                      {dv, s.v, 16, true},
                      {d_log_decay, s.gate, 4, true},
                      {d_beta, s.gate, 4, true},
                      {d_state_in, s.state, 16, true},
                      {workspace, need, 16, true}};
  if ((st = check_args(args, 15)) != RET_OK) return st;
  if (!workspace || workspace_bytes < need) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, 16)) != RET_OK) return st;
  DeltaParams p = params_of(desc, cu_seqlens, s, q, k, v, log_decay, beta, state_in);
  p.dout = dout;
  p.d_state_out = d_state_out;
  p.d_state_in = d_state_in;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.d_log_decay = d_log_decay;
  p.d_beta = d_beta;
  Carve c{static_cast<char*>(workspace)};
  carve_bwd(c, p, layout_of(desc, packed, total_tokens), desc, s);
  return ret::launch_delta_bwd(p, desc->dk, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

ret_status_t retention_delta_step(const ret_delta_desc_t* desc, const void* q, const void* k, const void* v,
                                  const float* log_decay, const float* beta, void* o, float* state,
                                  const int32_t* slots, int64_t num_slots, hipStream_t stream) {
  ret_status_t st = check_delta(desc, false, 0);
  if (st != RET_OK) return st;
  if (desc->seqlen != 1) return RET_ERR_SHAPE;
  if (num_slots < 1 || num_slots > INT32_MAX || (!slots && num_slots != desc->batch)) return RET_ERR_SHAPE;
  if (!q || !k || !v || !log_decay || !beta || !o || !state) return RET_ERR_NULL;
  const Sizes s = sizes_of(desc, false, 0);
  const size_t pool = (size_t)num_slots * desc->v_heads * desc->dk * desc->dv * sizeof(float);
  const Arg args[] = {{q, s.qk, 16, false},
                      {k, s.qk, 16, false},
                      {v, s.v, 16, false},
                      {log_decay, s.gate, 4, false},
                      {beta, s.gate, 4, false},
                      {slots, (size_t)desc->batch * sizeof(int32_t), 4, false},
                      {o, s.v, 16, true},
                      {state, pool, 16, true}};
  if ((st = check_args(args, 8)) != RET_OK) return st;
  ret::DeltaStepParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.log_decay = log_decay;
  p.beta = beta;
  p.o = o;
  p.state = state;
  p.slots = slots;
  p.batch = desc->batch;
  p.k_heads = desc->k_heads;
  p.heads = desc->v_heads;
  p.num_slots = (int)num_slots;
  p.scale = desc->scale;
  return ret::launch_delta_step(p, desc->dk, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

}  // extern "C"
