// kv_append_ex.hip -- the append with head norms, and of trees (kv_append.hpp).
#include "kv_append.hpp"

namespace effort {

hipError_t launch_append_ex(const AppendArgs& a, int32_t dtype, hipStream_t s) {
  return append_dtype<true>(a, dtype, s);
}

}  // namespace effort
