// kv_attend.hip -- causal attention over the paged 8-bit cache.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace effort {

constexpr int AT_T = 64;

// One wave per (new token, query head), in one pass over the visible tokens,
// 64 at a time: lane t's score of token t, the running maximum and sum, then
// each lane its elements of the weighted sum of values.
template <int DT, int FMT, int D>
__global__ __launch_bounds__(AT_T) void k_attend_rows(AttendArgs a) {
  typedef typename ElemOf<DT>::T T;
  const int lane = (int)threadIdx.x;
  const int32_t tok = (int32_t)blockIdx.x, head = (int32_t)blockIdx.y;
  int lo = 0, hi = a.b.seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start_of(a.b, mid) <= tok) lo = mid; else hi = mid;
  }
  const int32_t s0 = start_of(a.b, lo), s1 = start_of(a.b, lo + 1);
  if (tok < s0 || tok >= s1) return;
  const int64_t len = a.b.lens[lo], pos = len - (s1 - s0) + (tok - s0);
  const int64_t cap = (int64_t)a.b.max_pages * a.page_tokens;
  const int64_t first = a.window && pos + 1 > a.window ? pos + 1 - a.window : 0;
  const int64_t end = pos + 1 < cap ? pos + 1 : cap;
  const int kvh = head / (a.q_heads / a.kv_heads);
  __shared__ float q[D];
  __shared__ float p[AT_T];
  __shared__ int64_t base[AT_T];
  __shared__ float vscale[AT_T];
  const T* row = static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)head * D;
  for (int i = lane; i < D; i += AT_T) q[i] = (float)row[i];
  __syncthreads();
  float m = -INFINITY, l = 0.0f, acc[D / AT_T];
#pragma unroll
  for (int i = 0; i < D / AT_T; ++i) acc[i] = 0.0f;
  for (int64_t t0 = first; t0 < end; t0 += AT_T) {
    const int64_t t = t0 + lane;
    float s = -INFINITY;
    int64_t at = -1;
    if (t < end) {
      const int32_t page = a.b.table[lo * a.b.table_stride + t / a.page_tokens];
      if (page >= 0 && page < a.b.pages) {
        const int64_t ph = (int64_t)page * a.kv_heads + kvh;
        at = (ph * a.page_tokens + t % a.page_tokens) * D;
        float dot = 0.0f;
        for (int i = 0; i < D; ++i) dot = __builtin_fmaf(q[i], decode<FMT>(a.kc[at + i]), dot);
        const float ks = a.ks[ph], vs = a.vs[ph];
        s = dot * ks * a.scale;
        const bool bad = !(fabsf(ks) < INFINITY) || !(fabsf(vs) < INFINITY);
        if (bad) s = __uint_as_float(0x7FC00000u);
        vscale[lane] = bad ? 1.0f : vs;
      }
    }
    base[lane] = at;
    float top = at >= 0 ? s : -INFINITY;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float mn = fmaxf(m, top);
    // mn is -inf where nothing but NaN scores has been seen: they stay NaN
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float w = at >= 0 ? expf(s - ref) : 0.0f;
    p[lane] = w;
    __syncthreads();
    const float alpha = expf(m - ref);
    m = mn;
    float sum = w;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    l = l * alpha + sum;
#pragma unroll
    for (int i = 0; i < D / AT_T; ++i) acc[i] *= alpha;
    for (int j = 0; j < AT_T; ++j) {
      const int64_t b = base[j];
      if (b < 0) continue;
      const float pv = p[j] * vscale[j];
#pragma unroll
      for (int i = 0; i < D / AT_T; ++i)
        acc[i] = __builtin_fmaf(pv, decode<FMT>(a.vc[b + lane + i * AT_T]), acc[i]);
    }
    __syncthreads();
  }
  T* out = static_cast<T*>(a.out) + tok * a.out_stride + (int64_t)head * D;
#pragma unroll
  for (int i = 0; i < D / AT_T; ++i) out[lane + i * AT_T] = (T)(l == 0.0f ? 0.0f : acc[i] / l);
}

uint64_t attend_workspace(int32_t, int32_t, int32_t, int64_t, int32_t) { return 0; }

template <int DT, int FMT>
static hipError_t attend_dim(const AttendArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.b.tokens, (unsigned)a.q_heads);
  if (a.dim == 64)
    hipLaunchKernelGGL((k_attend_rows<DT, FMT, 64>), grid, dim3(AT_T), 0, s, a);
  else
    hipLaunchKernelGGL((k_attend_rows<DT, FMT, 128>), grid, dim3(AT_T), 0, s, a);
  return hipGetLastError();
}

template <int DT>
static hipError_t attend_fmt(const AttendArgs& a, hipStream_t s) {
  return a.format == EFFORT_KV_I8 ? attend_dim<DT, EFFORT_KV_I8>(a, s) : attend_dim<DT, EFFORT_KV_E4M3>(a, s);
}

hipError_t launch_attend(const AttendArgs& a, int32_t dtype, hipStream_t s) {
  switch (dtype) {
    case EFFORT_F32: return attend_fmt<EFFORT_F32>(a, s);
    case EFFORT_F16: return attend_fmt<EFFORT_F16>(a, s);
    case EFFORT_BF16: return attend_fmt<EFFORT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace effort
