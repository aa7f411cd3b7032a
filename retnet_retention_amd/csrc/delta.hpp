// Internal interface between the delta rule's C-ABI layer and its kernels:
// parameters, the workspace's layout and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ret {

constexpr int kDeltaBlock = 64;  // tokens of a block
constexpr int kDeltaGroup = 2;   // blocks between two fp32 copies of the state (backward)

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
  // per (block, head): T = (I + A)^-1 diag(beta) and M = P T in planes, in the backward
  // also the transposes of T and P; the decay vectors
  void *t, *m, *tt, *pt;
  // per (block, key head): keys by rows and by columns, queries by rows, in the
  // backward also by columns, in the order the lanes take them
  void *kf, *kc, *qf, *qc;
  float* vec;  // [4][64]: exp(G_r), exp(G_last - G_r), beta_r, unused
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
  void *snap, *dsnap;  // per (block, head): the state at the block's start and the state's gradient at its end, [dv][dk]
  float* anchor;       // per (group, head): the fp32 state at the group's end
  void* u;             // the written values V', [tokens][heads][d] in planes
  float *odo, *vdv, *udv;  // per (block, head, slice): row sums o.dO, v.dv, V'.dv
  float* adot;            // per (group, head, slice): <state, its gradient> at the group's end
};

// Sizes that the host needs to carve a workspace (T of `dtype`, head size d).
struct DeltaLayout {
  size_t blocks;  // numbered blocks
  size_t groups;
  size_t mat_plane;  // bytes of one 64 x 64 plane
  int planes;        // planes that hold an fp32 operand: 2 bf16 values, or 1 fp32
  int mat_planes;    // the same for the backward's matrices: 3, or 1
  int slices;        // workgroups that share a head's value columns
};
DeltaLayout delta_layout(int batch, int seqlen, int d, int dtype, bool packed, int total);

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
