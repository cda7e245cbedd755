// kv_attend_tree.hip -- attention of trees of new tokens over the cache (kv_attend.hpp).
#include "kv_attend.hpp"

namespace effort {

// Enough for any type and any table: two parts of each block, and the plan.
uint64_t tree_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads) {
  if (seqs == 0 || tokens == 0) return 0;
  const int32_t group = q_heads / kv_heads;
  const int rt = row_tiles(seqs, tokens, group);
  const int rows = rt ? 16 * rt : tree_rows(seqs, tokens, group) == 1 ? prompt_rows<1>() : prompt_rows<2>();
  return (uint64_t)split_blocks() * 2 * (uint64_t)(rows * (dim + 2)) * sizeof(float) + (rt ? 0 : sizeof(Plan));
}

hipError_t launch_attend_tree(const AttendArgs& a, int32_t dtype, hipStream_t s) {
  return attend_dtype<true>(a, dtype, s);
}

}  // namespace effort
