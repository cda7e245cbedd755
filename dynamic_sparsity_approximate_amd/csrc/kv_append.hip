// kv_append.hip -- rotation of queries and keys, and the append to the paged 8-bit cache.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace effort {

constexpr int AP_T = 256;

// ---------------------------------------------------------------- table

// Angles are reduced in double: at row 2^20 a float angle would be off by 0.03.
__global__ void k_rope_table(double base, int64_t rows, int half, float2* table) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows * half) return;
  const int64_t row = i / half;
  const int pair = (int)(i - row * half);
  double s, c;
  sincos((double)row * pow(base, -(double)pair / (double)half), &s, &c);
  table[i] = make_float2((float)c, (float)s);
}

hipError_t launch_rope_table(double base, int64_t rows, int32_t rot, float* table, hipStream_t s) {
  // row slices, so that a grid stays below 2^31 blocks
  const int half = rot / 2;
  const int64_t blocks = (rows * half + 255) / 256;
  if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_rope_table, dim3((unsigned)blocks), dim3(256), 0, s, base, rows, half,
                     reinterpret_cast<float2*>(table));
  return hipGetLastError();
}

// ---------------------------------------------------------------- append

// Four pairs of a head: where their elements are.  With `pairs` side by side
// (interleaved, or nothing to rotate) the chunk is 8 elements from `a`; else 4
// from `a` and 4 from `b`.
struct Chunk {
  int a, b, pair;  // pair: of the table, when rotated
  bool rotated, side;
};

__device__ inline Chunk chunk_of(int c, int dim, int rot, bool interleaved) {
  Chunk k;
  const int p = 4 * c;
  k.rotated = p < rot / 2;
  k.pair = p;
  k.side = interleaved || !k.rotated;
  if (interleaved) {
    k.a = 2 * p;
  } else if (k.rotated) {
    k.a = p;
  } else {
    k.a = rot + 2 * (p - rot / 2);
  }
  k.b = k.side ? k.a + 4 : p + rot / 2;
  return k;
}

// The chunk's elements in the order (first of a pair, second) x 4.
template <typename T>
__device__ inline void load_chunk(const T* row, const Chunk& k, bool interleaved, bool vec, float* x) {
  float a[4], b[4];
  load_n<4>(row + k.a, vec, a);
  load_n<4>(row + k.b, vec, b);
  if (k.rotated && interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = i < 2 ? a[2 * i] : b[2 * i - 4];
      x[4 + i] = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
}

// x (double) to the float that rounds to the same code: towards zero, with the
// last bit set if anything was cut off.  A later rounding to fewer bits, ties
// to even, then gives what rounding x at once would.
__device__ inline float round_to_odd(double x) {
  const float f = __double2float_rz(x);
  return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The chunk rotated; a key's products and sum are exact to 2^-53, so that its
// code is the nearest one even where the sum nearly cancels.
__device__ inline void rotate_exact(const float* x, const float2* cs, bool rotated, double* y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = x[i], b = x[4 + i];
    if (rotated) {
      const double c = cs[i].x, s = cs[i].y;
      y[i] = __builtin_fma(a, c, -(b * s));
      y[4 + i] = __builtin_fma(b, c, a * s);
    } else {
      y[i] = a;
      y[4 + i] = b;
    }
  }
}

// 1.f of the largest code and its exponent: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6.
template <int FMT>
__device__ inline int scale_exp(uint32_t amax_bits) {
  const uint32_t top = FMT == EFFORT_KV_I8 ? 0x7E0000u : 0x600000u;
  const int e = (int)(amax_bits >> 23) - 127 - (FMT == EFFORT_KV_I8 ? 6 : 8) +
                ((amax_bits & 0x7FFFFFu) > top ? 1 : 0);
  return e < EFFORT_KV_MIN_EXP ? EFFORT_KV_MIN_EXP : e;  // also for zero and subnormals
}

// Four codes of y, nearest, ties to even; |y| is at most the largest code.
template <int FMT>
__device__ inline uint32_t encode4(float y0, float y1, float y2, float y3) {
  if (FMT == EFFORT_KV_I8) {
    auto c = [](float y) { return (uint32_t)(int)__builtin_rintf(y) & 0xFFu; };
    return c(y0) | c(y1) << 8 | c(y2) << 16 | c(y3) << 24;
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, w, true);
}

// The rotation of one chunk's queries, rounded once in fp32.
__device__ inline void rotate_near(const float* x, const float2* cs, bool rotated, float* y) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = rotated ? __builtin_fmaf(x[j], cs[j].x, -(x[4 + j] * cs[j].y)) : x[j];
    y[4 + j] = rotated ? __builtin_fmaf(x[4 + j], cs[j].x, x[j] * cs[j].y) : x[4 + j];
  }
}

__device__ inline void load_rope(const float2* row, const Chunk& k, float2* cs) {
#pragma unroll
  for (int j = 0; j < 4; ++j) cs[j] = k.rotated ? row[k.pair + j] : make_float2(1.0f, 0.0f);
}

constexpr int AP_QH = 4;  // query heads of a thread: they share its cosines and sines

// One block per (page of a sequence, head, keys or values), then blocks of 256
// (token, 4 heads, chunk) items of the queries.  A page's block keeps its new
// elements in registers between the search for the largest magnitude and the
// codes: IT chunks a thread, up to a whole page.  A prompt is bound by its
// bytes (and read once), a single token by the chain starts -> page -> scale;
// the new rows are therefore asked for before the page is known.
template <int DT, int FMT, int IT>
__global__ __launch_bounds__(AP_T) void k_append(AppendArgs a, int32_t units, int32_t per_token,
                                                 int32_t kv_vec, int32_t q_vec) {
  typedef typename ElemOf<DT>::T T;
  const int tid = (int)threadIdx.x;
  const int dim = a.dim, cpr = dim / 8;
  const bool inter = a.interleaved != 0;
  const float2* rope = reinterpret_cast<const float2*>(a.rope);
  const int half = a.rot / 2;
  const int64_t kv_blocks = (int64_t)units * a.kv_heads * 2;

  if ((int64_t)blockIdx.x >= kv_blocks) {
    const int64_t i = ((int64_t)blockIdx.x - kv_blocks) * AP_T + tid;
    const int32_t per = (a.q_heads + AP_QH - 1) / AP_QH * cpr;
    const int64_t tok = i / per;
    if (tok >= a.b.tokens) return;
    int lo = 0, hi = a.b.seqs;  // the last sequence that starts at or before tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start_of(a.b, mid) <= tok) lo = mid; else hi = mid;
    }
    const int32_t s0 = start_of(a.b, lo), s1 = start_of(a.b, lo + 1);
    if (tok < s0 || tok >= s1) return;
    const int64_t pos = (int64_t)a.b.lens[lo] - (s1 - s0) + (tok - s0);
    if (pos < 0 || pos >= (int64_t)a.b.max_pages * a.page_tokens) return;
    const int r = (int)(i - tok * per), head = r / cpr * AP_QH;
    const Chunk k = chunk_of(r % cpr, dim, a.rot, inter);
    float2 cs[4];
    load_rope(rope + pos * half, k, cs);
    const T* row = static_cast<const T*>(a.q) + tok * a.q_stride + (int64_t)head * dim;
    T* out = static_cast<T*>(a.q_out) + tok * a.q_out_stride + (int64_t)head * dim;
    float x[AP_QH][8];
#pragma unroll
    for (int h = 0; h < AP_QH; ++h)
      if (head + h < a.q_heads) load_chunk(row + h * dim, k, inter, q_vec != 0, x[h]);
#pragma unroll
    for (int h = 0; h < AP_QH; ++h) {
      if (head + h >= a.q_heads) break;
      float y[8];
      rotate_near(x[h], cs, k.rotated, y);
      if (k.rotated && inter) {
        const float z[8] = {y[0], y[4], y[1], y[5], y[2], y[6], y[3], y[7]};
        store_n<4>(out + h * dim + k.a, q_vec != 0, z);
        store_n<4>(out + h * dim + k.b, q_vec != 0, z + 4);
      } else {
        store_n<4>(out + h * dim + k.a, q_vec != 0, y);
        store_n<4>(out + h * dim + k.b, q_vec != 0, y + 4);
      }
    }
    return;
  }

  const int32_t ph = (int32_t)((int64_t)blockIdx.x / units);
  const int32_t u = (int32_t)((int64_t)blockIdx.x - (int64_t)ph * units);
  const int head = ph >> 1;
  const bool is_k = (ph & 1) == 0;
  __shared__ int s_seq;
  __shared__ uint32_t s_max[AP_T / 64];
  const int32_t pt = a.page_tokens;
  // units before sequence i: one per token, or enough for the pages that its
  // tokens can touch (n / pt + 2)
  auto before = [&](int32_t i) {
    const int32_t t = start_of(a.b, i);
    return per_token ? t : t / pt + 2 * i;
  };
  int seq = 0;
  if (a.b.seqs > 1) {
    if (tid == 0) s_seq = a.b.seqs;
    __syncthreads();
    for (int i = tid; i < a.b.seqs; i += AP_T)
      if (before(i) <= u && u < before(i + 1)) atomicMin(&s_seq, i);
    __syncthreads();
    seq = s_seq;
    if (seq >= a.b.seqs) return;
  } else if (u < before(0) || u >= before(1)) {
    return;
  }
  const int32_t t0 = start_of(a.b, seq);
  const int64_t n = (int64_t)start_of(a.b, seq + 1) - t0, len = a.b.lens[seq];
  const int64_t pos0 = len - n, from = pos0 > 0 ? pos0 : 0;
  const int64_t pg = from / pt + (u - before(seq));
  if (n <= 0 || len <= 0 || pg >= a.b.max_pages) return;
  const int64_t lo = pg * pt > from ? pg * pt : from, hi = (pg + 1) * pt < len ? (pg + 1) * pt : len;
  if (lo >= hi) return;
  const int32_t page = a.b.table[seq * a.b.table_stride + pg];
  const int slot0 = (int)(lo - pg * pt), m = (int)(hi - lo);
  const int64_t tok0 = t0 + (lo - pos0);
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const T* rows = static_cast<const T*>(is_k ? a.k : a.v) + tok0 * stride + (int64_t)head * dim;
  const int rot = is_k ? a.rot : 0, items = m * cpr;
  const bool side = is_k && inter;

  float y[IT][8];  // the new elements, first rotated (round_to_odd), then coded
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = tid + it * AP_T, r = i / cpr;
    if (i < items) load_chunk(rows + r * stride, chunk_of(i - r * cpr, dim, rot, side), side, kv_vec != 0, y[it]);
  }
  if (page < 0 || page >= a.b.pages) return;
  uint8_t* codes = (is_k ? a.kc : a.vc) + ((int64_t)page * a.kv_heads + head) * pt * dim;
  float* scale = (is_k ? a.ks : a.vs) + (int64_t)page * a.kv_heads + head;
  const float old = *scale;

  uint32_t top = 0;  // as bits: a NaN is above an infinity, that above every number
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = tid + it * AP_T, r = i / cpr;
    if (i >= items) continue;
    const Chunk k = chunk_of(i - r * cpr, dim, rot, side);
    if (k.rotated) {
      float2 cs[4];
      double z[8];
      load_rope(rope + (lo + r) * half, k, cs);
      rotate_exact(y[it], cs, true, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[it][j] = round_to_odd(z[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(y[it][j]) & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  if ((tid & 63) == 0) s_max[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < AP_T / 64; ++w) top = s_max[w] > top ? s_max[w] : top;

  const bool fresh = slot0 == 0;
  float now = __uint_as_float((uint32_t)(scale_exp<FMT>(top) + 127) << 23);
  bool bad = top >= 0x7F800000u;
  if (!fresh) {
    bad = bad || (__float_as_uint(old) & 0x7F800000u) == 0x7F800000u;
    now = old > now ? old : now;
  }
  if (bad) now = __uint_as_float(0x7FC00000u);
  if (tid == 0) *scale = now;
  if (!fresh && now > old) {
    const double ratio = (double)old / (double)now;
    uint32_t* w = reinterpret_cast<uint32_t*>(codes);
    for (int i = tid; i < slot0 * dim / 4; i += AP_T) {
      const uint32_t c = w[i];
      float z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = round_to_odd((double)decode<FMT>(c >> (8 * j) & 0xFFu) * ratio);
      w[i] = encode4<FMT>(z[0], z[1], z[2], z[3]);
    }
  }
  // A power of two divides exactly.  By another scale (a cache that this
  // kernel did not begin) the elements are rotated again and divided in double.
  const bool pow2 = (__float_as_uint(now) & 0x7FFFFFu) == 0;
  const float per = (float)(1.0 / (double)now);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = tid + it * AP_T, r = i / cpr;
    if (i >= items) continue;
    const Chunk k = chunk_of(i - r * cpr, dim, rot, side);
    float* z = y[it];
    if (pow2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] *= per;
    } else if (!bad) {
      float x[8];
      float2 cs[4];
      double d[8];
      load_chunk(rows + r * stride, k, side, kv_vec != 0, x);
      load_rope(rope + (lo + r) * half, k, cs);
      rotate_exact(x, cs, k.rotated, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = round_to_odd(d[j] / (double)now);
    }
    uint32_t c[2] = {0, 0};
    if (!bad) {
      if (k.rotated && side) {
        c[0] = encode4<FMT>(z[0], z[4], z[1], z[5]);
        c[1] = encode4<FMT>(z[2], z[6], z[3], z[7]);
      } else {
        c[0] = encode4<FMT>(z[0], z[1], z[2], z[3]);
        c[1] = encode4<FMT>(z[4], z[5], z[6], z[7]);
      }
    }
    uint8_t* out = codes + (slot0 + r) * dim;
    *reinterpret_cast<uint32_t*>(out + k.a) = c[0];
    *reinterpret_cast<uint32_t*>(out + k.b) = c[1];
  }
}

template <int DT, int FMT, int IT>
static hipError_t append_it(const AppendArgs& a, hipStream_t s) {
  typedef typename ElemOf<DT>::T T;
  // units: pages that may receive tokens (fewer of the two bounds)
  const int64_t by_page = a.b.tokens / a.page_tokens + 2 * (int64_t)a.b.seqs;
  const int per_token = a.b.tokens <= by_page ? 1 : 0;
  const int64_t units = per_token ? a.b.tokens : by_page;
  const int64_t q_items = (int64_t)a.b.tokens * ((a.q_heads + AP_QH - 1) / AP_QH) * (a.dim / 8);
  const int64_t blocks = units * a.kv_heads * 2 + (q_items + AP_T - 1) / AP_T;
  if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
  const int kv_vec = rows_aligned<4, T>(a.k, a.k_stride) && rows_aligned<4, T>(a.v, a.v_stride);
  const int q_vec = a.q_heads && rows_aligned<4, T>(a.q, a.q_stride) && rows_aligned<4, T>(a.q_out, a.q_out_stride);
  hipLaunchKernelGGL((k_append<DT, FMT, IT>), dim3((unsigned)blocks), dim3(AP_T), 0, s, a, (int32_t)units,
                     per_token, kv_vec, q_vec);
  return hipGetLastError();
}

// Chunks of a page per thread: a page's rows, or the call's if those are fewer.
template <int DT, int FMT>
static hipError_t append_fmt(const AppendArgs& a, hipStream_t s) {
  const int64_t rows = a.b.tokens < a.page_tokens ? a.b.tokens : a.page_tokens;
  const int64_t it = (rows * (a.dim / 8) + AP_T - 1) / AP_T;
  if (it <= 1) return append_it<DT, FMT, 1>(a, s);
  if (it <= 2) return append_it<DT, FMT, 2>(a, s);
  if (it <= 4) return append_it<DT, FMT, 4>(a, s);
  return append_it<DT, FMT, 8>(a, s);
}

template <int DT>
static hipError_t append_launch(const AppendArgs& a, hipStream_t s) {
  return a.format == EFFORT_KV_I8 ? append_fmt<DT, EFFORT_KV_I8>(a, s) : append_fmt<DT, EFFORT_KV_E4M3>(a, s);
}

hipError_t launch_append(const AppendArgs& a, int32_t dtype, hipStream_t s) {
  switch (dtype) {
    case EFFORT_F32: return append_launch<EFFORT_F32>(a, s);
    case EFFORT_F16: return append_launch<EFFORT_F16>(a, s);
    case EFFORT_BF16: return append_launch<EFFORT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace effort
