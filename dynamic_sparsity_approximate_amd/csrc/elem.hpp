// elem.hpp -- device helpers on the element types of layer.hpp's kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "effort.h"
#include "layer.hpp"

namespace effort {

template <int DT>
struct ElemOf;
template <>
struct ElemOf<EFFORT_F32> {
  typedef float T;
};
template <>
struct ElemOf<EFFORT_F16> {
  typedef _Float16 T;
};
template <>
struct ElemOf<EFFORT_BF16> {
  typedef __bf16 T;
};

template <int N, typename T>
struct alignas(N * sizeof(T)) Vec {
  T e[N];
};

// N elements at p as floats; `vec`: p is aligned to them all.
template <int N, typename T>
__device__ inline void load_n(const T* p, bool vec, float* x) {
  if (vec) {
    const Vec<N, T> t = *reinterpret_cast<const Vec<N, T>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)t.e[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)p[i];
  }
}

// Rounds to nearest even, once.
template <int N, typename T>
__device__ inline void store_n(T* p, bool vec, const float* x) {
  if (vec) {
    Vec<N, T> t;
#pragma unroll
    for (int i = 0; i < N; ++i) t.e[i] = (T)x[i];
    *reinterpret_cast<Vec<N, T>*>(p) = t;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = (T)x[i];
  }
}

// Whether rows of T at p, `stride` elements apart, all start aligned to N elements.
template <int N, typename T>
inline bool rows_aligned(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) % (N * sizeof(T))) == 0 && stride % N == 0;
}

// q_starts[i], cut to [0, tokens].
__device__ inline int32_t start_of(const BatchArgs& b, int32_t i) {
  const int32_t t = b.starts[i];
  return t < 0 ? 0 : t > b.tokens ? b.tokens : t;
}

// The value of an 8-bit code before its scale.
template <int FMT>
__device__ inline float decode(uint32_t code) {
  if (FMT == EFFORT_KV_I8) return (float)(int32_t)(int8_t)code;
  return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

}  // namespace effort
