// C-ABI host layer of the norms around a token mixer: argument validation and
// launches on the caller's stream.
#include <cmath>

#include "host_checks.hpp"
#include "norms.hpp"

namespace {

using namespace ret_host;
using ret::NormParams;

ret_status_t check_norm(const ret_norm_desc_t* d) {
  if (!d) return RET_ERR_NULL;
  if (d->rows < 0 || d->rows > INT32_MAX || d->width < 1 || d->width > ret::kMaxNormWidth) return RET_ERR_SHAPE;
  if (d->dtype != RET_F32 && d->dtype != RET_BF16) return RET_ERR_UNSUPPORTED;
  if (!(std::isfinite(d->eps) && d->eps > 0.0f)) return RET_ERR_ARG;
  return RET_OK;
}

size_t row_bytes(const ret_norm_desc_t* d) { return (size_t)d->rows * d->width * elem_size(d->dtype); }
size_t weight_bytes(const ret_norm_desc_t* d) { return (size_t)d->width * sizeof(float); }

NormParams params_of(const ret_norm_desc_t* d) {
  NormParams p = {};
  p.rows = d->rows;
  p.width = d->width;
  p.center = d->center != 0;
  p.eps = d->eps;
  return p;
}

size_t sums_bytes(const ret_norm_desc_t* d, int sums) {
  if (check_norm(d) != RET_OK) return 0;
  return (size_t)sums * ret::norm_bwd_blocks(d->rows, d->width) * weight_bytes(d);
}

}  // namespace

extern "C" {

ret_status_t retention_head_norm_fwd(const ret_norm_desc_t* desc, const void* x, const float* weight,
                                     const void* gate, void* out, hipStream_t stream) {
  ret_status_t st = check_norm(desc);
  if (st != RET_OK) return st;
  if (desc->rows == 0) return RET_OK;
  if (!x || !out) return RET_ERR_NULL;
  const size_t n = row_bytes(desc);
  const Arg args[] = {{x, n, 16, false}, {weight, weight_bytes(desc), 16, false}, {gate, n, 16, false}, {out, n, 16, true}};
  if ((st = check_args(args, 4)) != RET_OK) return st;
  NormParams p = params_of(desc);
  p.x = x;
  p.weight = weight;
  p.gate = gate;
  p.out = out;
  return ret::launch_head_norm_fwd(p, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

size_t retention_head_norm_bwd_workspace_bytes(const ret_norm_desc_t* desc) { return sums_bytes(desc, 1); }

ret_status_t retention_head_norm_bwd(const ret_norm_desc_t* desc, const void* x, const float* weight,
                                     const void* gate, const void* dout, void* dx, float* dweight, void* dgate,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream) {
  ret_status_t st = check_norm(desc);
  if (st != RET_OK) return st;
  if ((weight == nullptr) != (dweight == nullptr)) return RET_ERR_NULL;
  if (desc->rows && (!x || !dout || !dx || (gate == nullptr) != (dgate == nullptr))) return RET_ERR_NULL;
  const size_t n = row_bytes(desc), nw = weight_bytes(desc), need = weight ? sums_bytes(desc, 1) : 0;
  const Arg args[] = {{x, n, 16, false},       {weight, nw, 16, false}, {gate, n, 16, false},
                      {dout, n, 16, false},    {dx, n, 16, true},       {dweight, nw, 16, true},
                      {dgate, n, 16, true},    {workspace, need, 16, true}};
  if ((st = check_args(args, 7)) != RET_OK) return st;
  if (need && (!workspace || workspace_bytes < need)) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, need ? 8 : 7)) != RET_OK) return st;
  NormParams p = params_of(desc);
  p.x = x;
  p.weight = weight;
  p.gate = gate;
  p.dout = dout;
  p.dx = dx;
  p.dweight = dweight;
  p.dgate = dgate;
  p.partial = static_cast<float*>(workspace);
  return ret::launch_head_norm_bwd(p, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

ret_status_t retention_residual_norm_fwd(const ret_norm_desc_t* desc, float skip, const void* x, const void* y,
                                         const float* weight, const float* post_weight, const float* scale, void* out,
                                         void* residual, hipStream_t stream) {
  ret_status_t st = check_norm(desc);
  if (st != RET_OK) return st;
  if (!std::isfinite(skip)) return RET_ERR_ARG;
  if (!weight) return RET_ERR_NULL;
  if (desc->rows == 0) return RET_OK;
  if (!x || !y || !out || !residual) return RET_ERR_NULL;
  const size_t n = row_bytes(desc), nw = weight_bytes(desc);
  const Arg args[] = {{x, n, 16, false},         {residual, n, 16, true},   {y, n, 16, false}, {weight, nw, 16, false},
                      {post_weight, nw, 16, false}, {scale, nw, 16, false}, {out, n, 16, true}};
  // a row of x is in registers before the row of the residual is written
  if ((st = check_args(args, 7, 0, 1)) != RET_OK) return st;
  NormParams p = params_of(desc);
  p.skip = skip;
  p.x = x;
  p.y = y;
  p.weight = weight;
  p.post = post_weight;
  p.scale = scale;
  p.out = out;
  p.residual = residual;
  return ret::launch_residual_norm_fwd(p, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

size_t retention_residual_norm_bwd_workspace_bytes(const ret_norm_desc_t* desc) { return sums_bytes(desc, 3); }

ret_status_t retention_residual_norm_bwd(const ret_norm_desc_t* desc, float skip, const void* x, const void* y,
                                         const float* weight, const float* post_weight, const float* scale,
                                         const void* dout, const void* dresidual, void* dx, void* dy, float* dweight,
                                         float* dpost_weight, float* dscale, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
  ret_status_t st = check_norm(desc);
  if (st != RET_OK) return st;
  if (!std::isfinite(skip)) return RET_ERR_ARG;
  if (!weight || !dweight || (post_weight == nullptr) != (dpost_weight == nullptr) ||
      (scale == nullptr) != (dscale == nullptr))
    return RET_ERR_NULL;
  if (desc->rows && (!x || !y || !dout || !dx || !dy)) return RET_ERR_NULL;
  const size_t n = row_bytes(desc), nw = weight_bytes(desc), need = sums_bytes(desc, 3);
  const Arg args[] = {{x, n, 16, false},           {y, n, 16, false},     {weight, nw, 16, false},
                      {post_weight, nw, 16, false}, {scale, nw, 16, false}, {dout, n, 16, false},
                      {dresidual, n, 16, false},   {dx, n, 16, true},     {dy, n, 16, true},
                      {dweight, nw, 16, true},     {dpost_weight, nw, 16, true}, {dscale, nw, 16, true},
                      {workspace, need, 16, true}};
  if ((st = check_args(args, 12)) != RET_OK) return st;
  if (need && (!workspace || workspace_bytes < need)) return RET_ERR_WORKSPACE;
  if ((st = check_args(args, need ? 13 : 12)) != RET_OK) return st;
  NormParams p = params_of(desc);
  p.skip = skip;
  p.x = x;
  p.y = y;
  p.weight = weight;
  p.post = post_weight;
  p.scale = scale;
  p.dout = dout;
  p.dresidual = dresidual;
  p.dx = dx;
  p.dy = dy;
  p.dweight = dweight;
  p.dpost = dpost_weight;
  p.dscale = dscale;
  p.partial = static_cast<float*>(workspace);
  return ret::launch_residual_norm_bwd(p, desc->dtype, stream) == hipSuccess ? RET_OK : RET_ERR_HIP;
}

}  // extern "C"
