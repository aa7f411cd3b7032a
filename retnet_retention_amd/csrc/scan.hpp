// Internal interface between the C-ABI layers of the gated recurrence and the
// short convolution and their kernels: parameters, workspaces, launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ret {

// Tiles of a batch's tokens are numbered over all of it: tile i of sequence b is b *
// (tiles of a sequence) + i, for packed sequences (row cu[b]) / tile + b + i, which no
// two sequences share.
inline int64_t tile_count(int batch, int seqlen, bool packed, int64_t total, int tile) {
  return packed ? total / tile + batch : (int64_t)batch * ((seqlen + (int64_t)tile - 1) / tile);
}

// The recurrence: tokens of a tile of the forward and of the backward. The states
// that the forward keeps stand before each of the backward's tiles. Long tiles make
// short chains, short ones leave less to wait for at a workgroup's begin and end. Calls in us,
//   forward, 256 and 128: 1 x 32768 x 1024 88 and 160, 1 x 131072 x 2560 542 and 870, 2 x 8192 x
//     4096 109 and 113, 4 x 2048 x 2560 with its inputs in the caches 39 and 36;
//   backward, 128 and 64: 1 x 32768 x 1024 172 and 320, 1 x 131072 x 2560 1170 and 1786, 2 x 8192
//     x 4096 191 and 205, 4 x 2048 x 2560 61 and 58.
constexpr int kScanTile = 256, kScanBwdTile = 128;
// Sequences of up to this many tokens may be one tile of the forward, of 1024 threads: then
// there is nothing to hand on, and nothing to clear before (scan_fwd.hip tells when).
constexpr int kScanOnly = 512;
// Channels of a workgroup: rows of 128 bytes in bf16, and a wave's lanes in the chain.
constexpr int kScanChannels = 64;

// What the workgroups of a call hand each other: a control block (word 1: errors),
// ticket counters 64 bytes apart, and a word for each tile and channel.
constexpr int kScanQueues = 16;
constexpr size_t kScanCtrlBytes = 64 * (1 + kScanQueues);
// whether any sequence has more than one tile of `tile` tokens
inline bool has_chain(int seqlen, bool packed, int64_t total, int tile) { return (packed ? total : seqlen) > tile; }

// Whether pairs of neighbouring elements of `size` bytes are aligned in every row.
inline bool pairs_aligned(const void* p, int64_t stride, int size) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (2 * size) == 0 && stride % 2 == 0);
}

struct ScanParams {
  const void *x, *decay, *gate;  // decay: log decays (fp32), or with `rate` what its sigmoid is taken of
  const float* rate;             // [width] or null
  const int* cu;                 // packed bounds or null
  int batch, seqlen, width, total, normalize;
  int64_t x_stride, decay_stride, gate_stride;  // elements from a token to the next
  void* o;
  const float* state_in;
  float* state_out;
  float* kept;     // [tiles of the backward][width], or null
  int* ctrl;
  uint64_t* hand;  // [tiles][width], or null: no sequence has two tiles
  int tiles;
  bool keep_error;  // the call's second launch: the control word stays
  // backward
  const void* dout;
  const float* d_state_out;
  float* d_state_in;
  void *dx, *ddecay, *dgate;
  float *drate, *partial;  // partial: [tiles][width] sums of drate
};
hipError_t launch_scan_fwd(const ScanParams& p, int dtype, hipStream_t stream);
hipError_t launch_scan_prep(const ScanParams& p, hipStream_t stream);  // the others' first step
hipError_t launch_scan_bwd(const ScanParams& p, int dtype, hipStream_t stream);

struct ScanStepParams {
  const void *x, *decay, *gate;
  const float* rate;
  void* o;
  float* state;
  const int* slots;  // state slot of each sequence, or null: its own index
  int batch, width, num_slots, normalize;
  int64_t x_stride, decay_stride, gate_stride;
};
hipError_t launch_scan_step(const ScanStepParams& p, int dtype, hipStream_t stream);

constexpr int kMinTaps = 2, kMaxTaps = 4;
struct ConvParams {
  const void* x;
  const float *weight, *bias;  // [width][taps], [width] or null
  const int* cu;
  int batch, seqlen, width, total, swish;
  int rows;  // backward: tokens of a wave
  int64_t x_stride;
  void* o;
  const void* state_in;  // [batch][taps - 1][width], oldest first
  void* state_out;
  int* ctrl;
  // backward
  const void *dout, *d_state_out;
  void *dx, *d_state_in;
  float *dweight, *dbias;
  float* partial;  // [blocks][taps + 1][width] sums of dweight and dbias
};
int64_t conv_bwd_blocks(int batch, int seqlen, int width, bool packed, int64_t total);
hipError_t launch_conv_fwd(const ConvParams& p, int taps, int dtype, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvParams& p, int taps, int dtype, hipStream_t stream);

struct ConvStepParams {
  const void* x;
  const float *weight, *bias;
  void *o, *state;
  const int* slots;
  int batch, width, num_slots, swish;
  int64_t x_stride;
};
hipError_t launch_conv_step(const ConvStepParams& p, int taps, int dtype, hipStream_t stream);

// ctrl[0] = 0, ctrl[1] = 2 if packed bounds leave the tensor or decrease, else 0
hipError_t launch_check_bounds(const int* cu, int batch, int total, int* ctrl, hipStream_t stream);

// Width limit of both: their launches count channels in groups of 64 or 128.
constexpr int kMaxScanWidth = 65536;

}  // namespace ret
