// Internal interface of the cache of parked states: parameters and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ret {

constexpr int kCacheBlock = 64;  // values that share a scale

struct StateCacheParams {
  float* state;       // [num_slots][values]; the write only reads it
  int8_t* codes;      // [cache_slots][values]
  float* scales;      // [cache_slots][blocks of a state]
  const int* at;      // [batch] cache slots
  const int* slots;   // [batch] slots of `state`, or null: the sequence's own index
  int batch;
  int64_t num_slots, cache_slots, values, blocks;
};
hipError_t launch_state_cache_write(const StateCacheParams& p, hipStream_t stream);
hipError_t launch_state_cache_read(const StateCacheParams& p, hipStream_t stream);

}  // namespace ret
