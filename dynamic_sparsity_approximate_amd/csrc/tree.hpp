// tree.hpp -- trees of new tokens (the parents of effort_kv_append_ex and its like), as the
// kernels walk them: from a token to its first ancestor, in LDS.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "effort.h"

namespace effort {

// An entry that is no earlier token of the sequence counts as none, so that every walk
// goes down and ends.
__device__ inline int16_t up_of(int32_t parent, int i) { return (int16_t)(parent >= 0 && parent < i ? parent : -1); }

// Whether n new tokens of a sequence, the first at position `pos`, are a tree: others have
// no place and see nothing.
__device__ inline bool is_tree(int64_t n, int64_t pos) { return n <= EFFORT_KV_MAX_TREE && pos >= 0; }

// Ancestors of token i.
__device__ inline int depth_of(const int16_t* up, int i) {
  int d = 0;
  for (int p = up[i]; p >= 0; p = up[p]) ++d;
  return d;
}

}  // namespace effort
