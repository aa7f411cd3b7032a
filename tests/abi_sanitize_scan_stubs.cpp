// Stand-ins for the launchers of the recurrence, the convolution and the cache of
// parked states in the sanitizer build of their C-ABI layer: they touch no device,
// check what the host layer hands them and count the calls.
#include "scan.hpp"
#include "state_cache.hpp"

extern "C" int launches;
int launches = 0;

namespace ret {
static hipError_t count(bool ok) {
  ++launches;
  return ok ? hipSuccess : hipErrorInvalidValue;
}
// one tile after another as the kernels number them, or one workgroup a sequence
static bool tiles_ok(const ScanParams& p, int tile) {
  const int64_t n = tile_count(p.batch, p.seqlen, p.cu, p.total, tile);
  return p.ctrl && p.tiles == n && (p.hand != nullptr) == has_chain(p.seqlen, p.cu, p.total, tile);
}
hipError_t launch_scan_fwd(const ScanParams& p, int, hipStream_t) {
  return count(tiles_ok(p, kScanTile) && (p.o || p.kept || !p.total) && p.x_stride >= p.width);
}
hipError_t launch_scan_bwd(const ScanParams& p, int, hipStream_t) {
  return count(tiles_ok(p, kScanBwdTile) && p.partial && p.kept && p.decay_stride >= p.width);
}
hipError_t launch_scan_step(const ScanStepParams& p, int, hipStream_t) { return count(p.num_slots > 0); }
int conv_bwd_rows(int64_t tokens, int width) { return tokens * width > 1 << 26 ? 128 : 16; }
int64_t conv_bwd_blocks(int batch, int seqlen, int width, bool packed, int64_t total) {
  return tile_count(batch, seqlen, packed, total, 4 * conv_bwd_rows(packed ? total : (int64_t)batch * seqlen, width));
}
hipError_t launch_conv_fwd(const ConvParams& p, int taps, int, hipStream_t) {
  return count((!p.cu || p.ctrl) && taps >= 2 && taps <= 4);
}
hipError_t launch_conv_bwd(const ConvParams& p, int, int, hipStream_t) { return count(p.ctrl && p.partial); }
hipError_t launch_conv_step(const ConvStepParams& p, int, int, hipStream_t) { return count(p.num_slots > 0); }
hipError_t launch_state_cache_write(const StateCacheParams& p, hipStream_t) {
  return count(p.blocks * kCacheBlock >= p.values && (p.blocks - 1) * kCacheBlock < p.values);
}
hipError_t launch_state_cache_read(const StateCacheParams& p, hipStream_t) { return count(p.at != nullptr); }
}  // namespace ret
