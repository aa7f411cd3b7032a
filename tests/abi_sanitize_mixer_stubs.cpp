// Stand-ins for the launchers and size functions of the delta rule and the norms
// in the sanitizer build of their C-ABI layer: they touch no device, check what
// the host layer hands them and count the calls.
#include "delta.hpp"
#include "norms.hpp"

extern "C" int launches;
int launches = 0;

namespace ret {
// as the kernels' own: two bf16 values (three for the backward's matrices) or one fp32
DeltaLayout delta_layout(int batch, int seqlen, int dtype, bool packed, int total) {
  DeltaLayout l;
  l.blocks = packed ? (size_t)total / kDeltaBlock + batch : ((size_t)seqlen + kDeltaBlock - 1) / kDeltaBlock * batch;
  l.planes = dtype == 1 ? 2 : 1;
  l.mat_planes = dtype == 1 ? 3 : 1;
  l.mat_plane = kDeltaBlock * kDeltaBlock * (dtype == 1 ? 2 : 4);
  return l;
}
static hipError_t count(bool ok) {
  ++launches;
  return ok ? hipSuccess : hipErrorInvalidValue;
}
hipError_t launch_delta_fwd(const DeltaParams& p, int, int, hipStream_t) {
  return count(p.ctrl && p.t && p.m && p.vec && p.kf && p.kc && p.qf);
}
hipError_t launch_delta_bwd(const DeltaParams& p, int, int dtype, hipStream_t) {
  return count(p.ctrl && p.t && p.vec && p.kf && p.kc && p.qc && p.pairs && p.tt && p.pt && p.snap && p.dsnap && p.u &&
               p.dv_rest && dtype >= 0);
}
hipError_t launch_delta_step(const DeltaStepParams& p, int, int, hipStream_t) { return count(p.num_slots > 0); }
int norm_bwd_blocks(int64_t rows, int width) {
  const int64_t rpb = width > 2048 ? 1 : 32;
  const int64_t need = (rows + rpb - 1) / rpb;
  return (int)(need < 1 ? 1 : need < 1024 ? need : 1024);
}
hipError_t launch_head_norm_fwd(const NormParams& p, int, hipStream_t) { return count(p.x && p.out); }
hipError_t launch_head_norm_bwd(const NormParams& p, int, hipStream_t) { return count(!p.dweight || p.partial); }
hipError_t launch_residual_norm_fwd(const NormParams& p, int, hipStream_t) { return count(p.residual); }
hipError_t launch_residual_norm_bwd(const NormParams& p, int, hipStream_t) { return count(p.partial); }
}  // namespace ret
