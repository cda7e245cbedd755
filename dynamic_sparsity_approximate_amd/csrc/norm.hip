// norm.hip -- norm after a block, gate, residual sum, norm before the next block.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace effort {

constexpr int NM_T = 1024;  // threads of a row at most

template <int CTRL>
__device__ inline float dpp_add(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true);
  return x + __int_as_float(y);
}

// The sum over a wave, in every lane: rotations within 16 lanes, then two exchanges.
__device__ inline float wave_sum(float x) {
  x = dpp_add<0x128>(x);  // row_ror 8, 4, 2, 1
  x = dpp_add<0x124>(x);
  x = dpp_add<0x122>(x);
  x = dpp_add<0x121>(x);
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The sum over the block; `red` is used once per kernel.
__device__ inline float block_sum(float x, float* red) {
  x = wave_sum(x);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  const int lane = (int)threadIdx.x & 63;
  return wave_sum(lane < waves ? red[lane] : 0.0f);
}

// Elements of one 16-byte load of the narrower type.
template <int DT>
constexpr int norm_width() {
  return DT == EFFORT_F32 ? 4 : 8;
}

// A thread's E elements of part c of a row: pieces of V that memory aligns, all
// threads' pieces side by side.  V divides n, so that a piece is in the row or not.
template <int V>
__device__ inline int piece_at(int c, int h, int pieces) {
  return ((c * pieces + h) * (int)blockDim.x + (int)threadIdx.x) * V;
}
template <int E, int V, typename T>
__device__ inline void load_part(const T* p, int c, int n, float* x) {
#pragma unroll
  for (int h = 0; h < E / V; ++h) {
    const int i = piece_at<V>(c, h, E / V);
    if (i < n) load_n<V>(p + i, true, x + h * V);
  }
}

template <int E, int V, typename T>
__device__ inline void store_part(T* p, int c, int n, const float* x) {
#pragma unroll
  for (int h = 0; h < E / V; ++h) {
    const int i = piece_at<V>(c, h, E / V);
    if (i < n) store_n<V>(p + i, true, x + h * V);
  }
}

// One block per row, the row in registers: NC parts of E elements a thread.
// Everything that the outputs need is loaded before the first sum, so that a
// single row costs one trip to memory and two exchanges over the block (4096 fp32
// elements: 2.5 us); for many rows the kernel moves each byte once and is bound
// by that (8191 bf16 rows of 4096 with both norms and a gate: 52 us, 5.2 TB/s).
// Rows of odd widths are read two or one element at a time, neighbouring threads
// side by side (1248 bf16 rows of 3282: 15.5 us; with a thread's eight elements
// side by side 39.6).
template <int DT, int RT, int NC, int V>
__global__ __launch_bounds__(NM_T) void k_norm(NormArgs a) {
  typedef typename ElemOf<DT>::T T;
  typedef typename ElemOf<RT>::T R;
  constexpr int E = norm_width<DT>();
  __shared__ float red[2][NM_T / 64];
  const int64_t row = blockIdx.x;
  const int n = (int)a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const R* resid = a.resid ? static_cast<const R*>(a.resid) + row * a.resid_stride : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_stride : nullptr;
  const T* post = static_cast<const T*>(a.post_w);
  const T* pre = static_cast<const T*>(a.pre_w);
  const float inv_n = 1.0f / (float)n;
  float r[NC][E], old[NC][E], w[NC][E];
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int k = 0; k < E; ++k) r[c][k] = old[c][k] = 0.0f, w[c][k] = a.scale;
    load_part<E, V>(x, c, n, r[c]);
    if (resid) load_part<E, V>(resid, c, n, old[c]);
    if (post) {
      float p[E] = {};
      load_part<E, V>(post, c, n, p);
#pragma unroll
      for (int k = 0; k < E; ++k) w[c][k] *= p[k];
    }
    if (gate) {
      float p[E] = {};
      load_part<E, V>(gate, c, n, p);
#pragma unroll
      for (int k = 0; k < E; ++k) w[c][k] *= p[k];
    }
#pragma unroll
    for (int k = 0; k < E; ++k) s = __builtin_fmaf(r[c][k], r[c][k], s);
  }
  const float rx = post ? 1.0f / sqrtf(block_sum(s, red[0]) * inv_n + a.eps) : 1.0f;
  s = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < E; ++k) {
      r[c][k] = __builtin_fmaf(r[c][k] * rx, w[c][k], old[c][k]);
      s = __builtin_fmaf(r[c][k], r[c][k], s);
    }
  if (a.resid_out) {
    R* to = static_cast<R*>(a.resid_out) + row * a.resid_out_stride;
#pragma unroll
    for (int c = 0; c < NC; ++c) store_part<E, V>(to, c, n, r[c]);
  }
  if (!a.out) return;
  float p[NC][E];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int k = 0; k < E; ++k) p[c][k] = 1.0f;
    if (pre) load_part<E, V>(pre, c, n, p[c]);
  }
  const float rr = 1.0f / sqrtf(block_sum(s, red[1]) * inv_n + a.eps);
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int k = 0; k < E; ++k) r[c][k] = r[c][k] * rr * p[c][k];
    store_part<E, V>(out, c, n, r[c]);
  }
}

// Rows too long for the registers of a block: read once for each sum and once
// more for the outputs.
template <int DT, int RT>
__global__ __launch_bounds__(NM_T) void k_norm_long(NormArgs a) {
  typedef typename ElemOf<DT>::T T;
  typedef typename ElemOf<RT>::T R;
  __shared__ float red[2][NM_T / 64];
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
    rx = 1.0f / sqrtf(block_sum(s, red[0]) * inv_n + a.eps);
  }
  auto value = [&](int64_t i) {
    float w = a.scale;
    if (post) w *= (float)post[i];
    if (gate) w *= (float)gate[i];
    return __builtin_fmaf((float)x[i] * rx, w, resid ? (float)resid[i] : 0.0f);
  };
  float rr = 1.0f;
  if (a.out) {
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.n; i += NM_T) {
      const float r = value(i);
      s = __builtin_fmaf(r, r, s);
    }
    rr = 1.0f / sqrtf(block_sum(s, red[1]) * inv_n + a.eps);
  }
  R* resid_out = a.resid_out ? static_cast<R*>(a.resid_out) + row * a.resid_out_stride : nullptr;
  T* out = a.out ? static_cast<T*>(a.out) + row * a.out_stride : nullptr;
  for (int64_t i = threadIdx.x; i < a.n; i += NM_T) {
    const float r = value(i);
    if (resid_out) resid_out[i] = (R)r;
    if (out) out[i] = (T)(pre ? r * rr * (float)pre[i] : r * rr);
  }
}

// Whether every row allows pieces of V elements.
template <int V, typename T, typename R>
static bool norm_aligned(const NormArgs& a) {
  return a.n % V == 0 && rows_aligned<V, T>(a.x, a.x_stride) &&
         (!a.resid || rows_aligned<V, R>(a.resid, a.resid_stride)) &&
         (!a.resid_out || rows_aligned<V, R>(a.resid_out, a.resid_out_stride)) &&
         (!a.out || rows_aligned<V, T>(a.out, a.out_stride)) &&
         (!a.gate || rows_aligned<V, T>(a.gate, a.gate_stride)) && rows_aligned<V, T>(a.post_w, 0) &&
         rows_aligned<V, T>(a.pre_w, 0);
}

template <int DT, int RT, int V>
static hipError_t norm_short(const NormArgs& a, hipStream_t s) {
  constexpr int E = norm_width<DT>(), NC_MAX = 32 / E;
  const int64_t parts = (a.n + E - 1) / E;
  // As many threads as there are parts, up to NM_T: with 16 elements a thread
  // one fp32 row of 4096 takes 4.7 us in a graph instead of 4.0, 8191 bf16 rows
  // 57.2 instead of 54.2.
  int nc = 1;
  while (parts > (int64_t)nc * NM_T) nc *= 2;
  const dim3 grid((unsigned)a.rows), block((unsigned)(((parts + nc - 1) / nc + 63) / 64 * 64));
  switch (nc) {
    case 1: hipLaunchKernelGGL((k_norm<DT, RT, 1, V>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_norm<DT, RT, 2, V>), grid, block, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_norm<DT, RT, 4, V>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((k_norm<DT, RT, NC_MAX, V>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <int DT, int RT>
static hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  typedef typename ElemOf<DT>::T T;
  typedef typename ElemOf<RT>::T R;
  constexpr int E = norm_width<DT>();
  if (a.n > 32 * NM_T) {
    hipLaunchKernelGGL((k_norm_long<DT, RT>), dim3((unsigned)a.rows), dim3(NM_T), 0, s, a);
    return hipGetLastError();
  }
  if (norm_aligned<E, T, R>(a)) return norm_short<DT, RT, E>(a, s);
  return norm_aligned<2, T, R>(a) ? norm_short<DT, RT, 2>(a, s) : norm_short<DT, RT, 1>(a, s);
}

// A launch has less than 2^32 threads: rows are taken so many at a time.
constexpr int64_t NM_ROWS = 0xFFFFFFFFll / NM_T;

template <int DT, int RT>
static hipError_t norm_rows(NormArgs a, hipStream_t s) {
  typedef typename ElemOf<DT>::T T;
  typedef typename ElemOf<RT>::T R;
  for (int64_t left = a.rows; left > 0; left -= NM_ROWS) {
    a.rows = left < NM_ROWS ? left : NM_ROWS;
    const hipError_t e = norm_launch<DT, RT>(a, s);
    if (e != hipSuccess) return e;
    a.x = static_cast<const T*>(a.x) + a.rows * a.x_stride;
    if (a.resid) a.resid = static_cast<const R*>(a.resid) + a.rows * a.resid_stride;
    if (a.gate) a.gate = static_cast<const T*>(a.gate) + a.rows * a.gate_stride;
    if (a.resid_out) a.resid_out = static_cast<R*>(a.resid_out) + a.rows * a.resid_out_stride;
    if (a.out) a.out = static_cast<T*>(a.out) + a.rows * a.out_stride;
  }
  return hipSuccess;
}

hipError_t launch_norm(const NormArgs& a, int32_t dtype, int32_t resid_dtype, hipStream_t s) {
  const bool f32 = resid_dtype == EFFORT_F32;
  switch (dtype) {
    case EFFORT_F32: return norm_rows<EFFORT_F32, EFFORT_F32>(a, s);
    case EFFORT_F16:
      return f32 ? norm_rows<EFFORT_F16, EFFORT_F32>(a, s) : norm_rows<EFFORT_F16, EFFORT_F16>(a, s);
    case EFFORT_BF16:
      return f32 ? norm_rows<EFFORT_BF16, EFFORT_F32>(a, s) : norm_rows<EFFORT_BF16, EFFORT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace effort
