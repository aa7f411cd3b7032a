// Argument checks shared by the C-ABI entry points (host only).
#pragma once

#include <cstddef>
#include <cstdint>

#include "retention.h"

namespace ret_host {

constexpr size_t kWsAlign = 256;
inline size_t align_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t elem_size(int32_t dtype) { return dtype == RET_BF16 ? 2 : 4; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// One pointer argument: its size, the alignment it needs, whether the call
// writes it.
struct Arg {
  const void* p;
  size_t bytes;
  size_t align;
  bool written;
};

// Every given pointer is aligned, and no written buffer overlaps another one
// (a pair listed in `same` may be exactly equal).
inline ret_status_t check_args(const Arg* a, int n, int same_i = -1, int same_j = -1) {
  for (int i = 0; i < n; ++i)
    if (a[i].p && reinterpret_cast<uintptr_t>(a[i].p) % a[i].align != 0) return RET_ERR_ALIGN;
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!a[i].written && !a[j].written) continue;
      if (i == same_i && j == same_j && a[i].p == a[j].p) continue;
      if (overlaps(a[i].p, a[i].bytes, a[j].p, a[j].bytes)) return RET_ERR_ALIAS;
    }
  return RET_OK;
}

}  // namespace ret_host
