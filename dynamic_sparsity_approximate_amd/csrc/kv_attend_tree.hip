// kv_attend_tree.hip -- attention of trees of new tokens over the cache (kv_attend.hpp).
#include "kv_attend.hpp"

namespace effort {

hipError_t launch_attend_tree(const AttendArgs& a, int32_t dtype, hipStream_t s) {
  return attend_dtype<true>(a, dtype, s);
}

}  // namespace effort
