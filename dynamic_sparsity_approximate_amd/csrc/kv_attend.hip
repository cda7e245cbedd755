// kv_attend.hip -- causal attention over the cache (kv_attend.hpp), and its workspace.
#include "kv_attend.hpp"

namespace effort {

// Enough for any type and any table.
uint64_t attend_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads) {
  if (seqs == 0 || tokens == 0) return 0;
  const int32_t group = q_heads / kv_heads;
  const int rt = row_tiles(seqs, tokens, group);
  if (rt) return (uint64_t)split_blocks() * 2 * (uint64_t)(16 * rt * (dim + 2)) * sizeof(float);
  uint64_t most = 0;
  for (int r = 1; r <= 2; ++r) {
    const PromptShape p = prompt_of(r, kv_heads, dim, seqs, tokens, group);
    const uint64_t rows = (uint64_t)p.tiles * kv_heads * p.splits * (64 * r);
    const uint64_t n = p.splits == 1 ? 0 : rows * (dim + 2) * sizeof(float);
    most = n > most ? n : most;
  }
  return most;
}

hipError_t launch_attend(const AttendArgs& a, int32_t dtype, hipStream_t s) { return attend_dtype<false>(a, dtype, s); }

}  // namespace effort
