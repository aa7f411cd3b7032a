// Internal interface between the delta rule's C-ABI layer and its kernels:
// parameters, the workspace's layout and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ret {

constexpr int kDeltaBlock = 64;  // tokens of a block

// Pointers into one call's workspace and the caller's tensors. Blocks are
// numbered over the whole batch: block i of sequence b is b * blocks_max + i,
// for packed sequences (row cu[b]) / 64 + b + i, which no two sequences share.
struct DeltaParams {
  const void *q, *k, *v;
  const float *log_decay, *beta;
  const int* cu;  // packed bounds or null
  int batch, seqlen, k_heads, heads, total, blocks_max;
  float scale;
  int* ctrl;
  // per (block, head): T = (I + A)^-1 diag(beta) in planes and the decay vectors; in
  // the forward also M = P T, in the backward the transposes of T and P
  void *t, *m, *tt, *pt;
  float* vec;  // [4][64]: exp(G_r), exp(G_last - G_r), beta_r, unused
  // per (block, key head): keys by rows and by columns, in the forward queries by
  // rows, in the backward by columns, in the order the lanes take them
  void *kf, *kc, *qf, *qc;
  float* pairs;  // backward, per (block, key head): [2][64][64] of q_r . k_s and k_r . k_s, s <= r
  // forward
  void* o;
  const float* state_in;
  float* state_out;
  // backward
  const void* dout;
  const float* d_state_out;
  float* d_state_in;
  void *dq, *dk, *dv;
  float *d_log_decay, *d_beta;
  // per (block, head), in planes: the state at the block's start and the state's
  // gradient at its end, [dv][dk]
  void *snap, *dsnap;
  void* u;        // the written values V', [tokens][heads][d] in planes
  void* dv_rest;  // what dv's own type leaves of it, [tokens][heads][d] (bf16)
};

// Sizes that the host needs to carve a workspace (T of `dtype`).
struct DeltaLayout {
  size_t blocks;  // numbered blocks
  size_t mat_plane;  // bytes of one 64 x 64 plane
  int planes;        // planes that hold an fp32 operand: 2 bf16 values, or 1 fp32
  int mat_planes;    // the same for the backward's matrices: 3, or 1
};
DeltaLayout delta_layout(int batch, int seqlen, int dtype, bool packed, int total);

hipError_t launch_delta_fwd(const DeltaParams& p, int d, int dtype, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaParams& p, int d, int dtype, hipStream_t stream);

struct DeltaStepParams {
  const void *q, *k, *v;
  const float *log_decay, *beta;
  void* o;
  float* state;
  const int* slots;  // state slot of each sequence, or null: its own index
  int batch, k_heads, heads, num_slots;
  float scale;
};
hipError_t launch_delta_step(const DeltaStepParams& p, int d, int dtype, hipStream_t stream);

}  // namespace ret
