// norm.hip -- norm after a block, gate, residual sum, norm before the next block.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace effort {

constexpr int NM_T = 256;

__device__ inline float block_sum(float x, float* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < NM_T / 64; ++w) t += red[w];
  return t;
}

// One block per row; the row is read once for each of its sums and once more
// for the outputs (after the first time from the caches).
template <int DT, int RT>
__global__ __launch_bounds__(NM_T) void k_norm(NormArgs a) {
  typedef typename ElemOf<DT>::T T;
  typedef typename ElemOf<RT>::T R;
  __shared__ float red[NM_T / 64];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const R* resid = a.resid ? static_cast<const R*>(a.resid) + row * a.resid_stride : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_stride : nullptr;
  const T* post = static_cast<const T*>(a.post_w);
  const T* pre = static_cast<const T*>(a.pre_w);
  const float inv_n = 1.0f / (float)a.n;
  float rx = 1.0f;
  if (post) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.n; i += NM_T) s = __builtin_fmaf((float)x[i], (float)x[i], s);
    rx = 1.0f / sqrtf(block_sum(s, red) * inv_n + a.eps);
  }
  auto value = [&](int64_t i) {
    float t = (float)x[i];
    if (post) t = t * rx * (float)post[i];
    if (gate) t *= (float)gate[i];
    t *= a.scale;
    return resid ? (float)resid[i] + t : t;
  };
  float rr = 1.0f;
  if (a.out) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.n; i += NM_T) {
      const float r = value(i);
      s = __builtin_fmaf(r, r, s);
    }
    rr = 1.0f / sqrtf(block_sum(s, red) * inv_n + a.eps);
  }
  R* resid_out = a.resid_out ? static_cast<R*>(a.resid_out) + row * a.resid_out_stride : nullptr;
  T* out = a.out ? static_cast<T*>(a.out) + row * a.out_stride : nullptr;
  for (int64_t i = threadIdx.x; i < a.n; i += NM_T) {
    const float r = value(i);
    if (resid_out) resid_out[i] = (R)r;
    if (out) out[i] = (T)(pre ? r * rr * (float)pre[i] : r * rr);
  }
}

template <int DT, int RT>
static hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm<DT, RT>), dim3((unsigned)a.rows), dim3(NM_T), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, int32_t dtype, int32_t resid_dtype, hipStream_t s) {
  const bool f32 = resid_dtype == EFFORT_F32;
  switch (dtype) {
    case EFFORT_F32: return norm_launch<EFFORT_F32, EFFORT_F32>(a, s);
    case EFFORT_F16:
      return f32 ? norm_launch<EFFORT_F16, EFFORT_F32>(a, s) : norm_launch<EFFORT_F16, EFFORT_F16>(a, s);
    case EFFORT_BF16:
      return f32 ? norm_launch<EFFORT_BF16, EFFORT_F32>(a, s) : norm_launch<EFFORT_BF16, EFFORT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace effort
