// kv_append.hip -- table of rotations; the append without head norms and trees (kv_append.hpp).
#include "kv_append.hpp"

namespace effort {

// ---------------------------------------------------------------- table

// Angles are reduced in double: at row 2^20 a float angle would be off by 0.03.
__global__ void k_rope_table(double base, int64_t first, int64_t rows, int half, float2* table) {
  const int64_t i = first + (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows * half) return;
  const int64_t row = i / half;
  const int pair = (int)(i - row * half);
  double s, c;
  sincos((double)row * pow(base, -(double)pair / (double)half), &s, &c);
  table[i] = make_float2((float)c, (float)s);
}

hipError_t launch_rope_table(double base, int64_t rows, int32_t rot, float* table, hipStream_t s) {
  const int half = rot / 2;
  const int64_t total = rows * half;
  constexpr int64_t most = 1ll << 31;  // entries of a launch, which has less than 2^32 threads
  for (int64_t first = 0; first < total; first += most) {
    const int64_t n = total - first < most ? total - first : most;
    hipLaunchKernelGGL(k_rope_table, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, base, first, rows, half,
                       reinterpret_cast<float2*>(table));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_append(const AppendArgs& a, int32_t dtype, hipStream_t s) {
  return append_dtype<false>(a, dtype, s);
}

}  // namespace effort
