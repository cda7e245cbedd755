// kv_append.hip -- rotation of queries and keys, and the append to the paged 8-bit cache.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "layer.hpp"

namespace effort {

constexpr int AP_T = 256;

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

// ---------------------------------------------------------------- append

// Pairs of a chunk (seven bf16 prompts, 6943 tokens in all, 32 and 8 heads: 50 us; 8 pairs take 61 to 73).
constexpr int CP = 4;

// CP pairs of a head: where their elements are.  With the pairs side by side
// (interleaved, or nothing to rotate) the chunk is 2 CP elements from `a`; else
// CP from `a` and CP from `b`.
struct Chunk {
  int a, b, pair;  // pair: of the table, when rotated
  bool rotated, side;
};

__device__ inline Chunk chunk_of(int c, int rot, bool interleaved) {
  Chunk k;
  const int p = CP * c;
  k.rotated = p < rot / 2;
  k.pair = p;
  k.side = interleaved || !k.rotated;
  k.a = k.side ? 2 * p : p;
  k.b = k.side ? k.a + CP : p + rot / 2;
  return k;
}

// The chunk's elements in memory's order: two halves, or (`together`, a choice
// of the whole block) one piece (interleaved pairs of the prompts above: 46 us,
// in halves 62).  `vec`: elements that rows are aligned to.
template <typename T>
__device__ inline void load_chunk(const T* row, const Chunk& k, bool together, int vec, float* y) {
  if (together) {
    load_n<2 * CP>(row + k.a, true, y);
  } else {
    load_n<CP>(row + k.a, vec >= CP, y);
    load_n<CP>(row + k.b, vec >= CP, y + CP);
  }
}

// ... the first of each pair and then the second ...
__device__ inline void from_order(bool pairs, float* y) {
  if (!pairs) return;
  const float a[2 * CP] = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
#pragma unroll
  for (int i = 0; i < CP; ++i) {
    y[i] = a[2 * i];
    y[CP + i] = a[2 * i + 1];
  }
}

// ... and back into their order in memory.
__device__ inline void to_order(const float* x, bool pairs, float* y) {
  if (pairs) {
#pragma unroll
    for (int i = 0; i < CP; ++i) {
      y[2 * i] = x[i];
      y[2 * i + 1] = x[CP + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * CP; ++i) y[i] = x[i];
  }
}

// x (double) to the float that rounds to the same code: the nearest one, and if
// that is inexact and its last bit 0, the neighbour on x's side (its last bit is
// 1).  A later rounding to fewer bits, ties to even, then gives what rounding x
// at once would: only an exact value can still look like a tie.
__device__ inline float round_to_odd(double x) {
  const float f = (float)x;
  const double rest = x - (double)f;  // exact; NaN for an infinite x, -+inf where f overflowed
  const int32_t bits = __float_as_int(f);
  const int32_t step = f == 0.0f || (rest > 0.0) == (f > 0.0f) ? 1 : -1;
  return (rest > 0.0 || rest < 0.0) && (bits & 1) == 0 ? __int_as_float(bits + step) : f;
}

// The chunk rotated; a key's products and sum are exact to 2^-53, so that its
// code is the nearest one even where the sum nearly cancels.
__device__ inline void rotate_exact(const float* x, const float2* cs, double* y) {
#pragma unroll
  for (int i = 0; i < CP; ++i) {
    const double a = x[i], b = x[CP + i], c = cs[i].x, s = cs[i].y;
    y[i] = __builtin_fma(a, c, -(b * s));
    y[CP + i] = __builtin_fma(b, c, a * s);
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

// The rotation of one chunk's queries in fp32: one product and the sum are
// rounded, 2^-24 of each.  The scores they go into are sums of fp32 products
// anyway; only codes, where the nearest one is promised, are worth double.
__device__ inline void rotate_near(const float* x, const float2* cs, float* y) {
#pragma unroll
  for (int j = 0; j < CP; ++j) {
    y[j] = __builtin_fmaf(x[j], cs[j].x, -(x[CP + j] * cs[j].y));
    y[CP + j] = __builtin_fmaf(x[CP + j], cs[j].x, x[j] * cs[j].y);
  }
}

// A chunk's cosines and sines.
__device__ inline void load_rope(const float2* at, float2* cs) {
#pragma unroll
  for (int j = 0; j < CP; ++j) cs[j] = at[j];
}

// Query heads of a thread: they share its cosines and sines (the prompts above:
// 50 us; with two heads 78, with one 139).
constexpr int AP_QH = 4;

// One block per (page of a sequence, head, keys or values), then blocks of four
// waves of the queries: a page's block waits most of its time, so those start
// first (spread evenly among the queries' blocks: 54.3 us instead of 50.1).  A
// page's block keeps its new elements in registers between the search for the
// largest magnitude and the codes: IT chunks a thread, up to a whole page.  A
// prompt (3.2 TB/s) waits for its bytes and for the rotation: caches warm, 44 us,
// without rotation 30; of those 14 the keys, in double, have 5 and the queries,
// whose blocks have the registers of a page's, 9.  A single token (4.1 us) waits
// for the chain starts -> page -> scale; the new rows are therefore asked for
// before the page is known.
template <int DT, int FMT, int IT>
__global__ __launch_bounds__(AP_T) void k_append(AppendArgs a, uint32_t first, int32_t units, int32_t per_token,
                                                 int32_t kv_vec, int32_t q_vec) {
  typedef typename ElemOf<DT>::T T;
  const int tid = (int)threadIdx.x;
  const int dim = a.dim, cpr_log = __builtin_ctz(dim / (2 * CP));  // chunks of a row: a power of two
  const bool inter = a.interleaved != 0;
  const float2* rope = reinterpret_cast<const float2*>(a.rope);
  const int half = a.rot / 2;
  const uint32_t kv_blocks = (uint32_t)units * (uint32_t)a.kv_heads * 2;
  const uint32_t block = first + blockIdx.x;

  if (block >= kv_blocks) {
    // a wave has 64 / chunks of a row * AP_QH heads of one token: all that leads
    // to its place is scalar (looked up by every lane, it took as long as the rest)
    const uint32_t slots = 64u >> cpr_log, per_wave = slots * AP_QH;
    const uint32_t parts = ((uint32_t)a.q_heads + per_wave - 1) / per_wave;  // waves of a token
    const uint32_t w = (block - kv_blocks) * (AP_T / 64) +
                       (uint32_t)__builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t tok = (int32_t)(w / parts);
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
    const uint32_t lane = (uint32_t)tid & 63;
    const uint32_t head0 = (w - (uint32_t)tok * parts) * per_wave + (lane >> cpr_log);
    const Chunk k = chunk_of((int)(lane & ((1u << cpr_log) - 1)), a.rot, inter);
    const T* row = static_cast<const T*>(a.q) + (int64_t)tok * a.q_stride;
    T* out = static_cast<T*>(a.q_out) + (int64_t)tok * a.q_out_stride;
    auto at = [&](int h) { return (head0 + (uint32_t)h * slots) * (uint32_t)dim; };  // the h-th of the lane's heads
    auto has = [&](int h) { return head0 + (uint32_t)h * slots < (uint32_t)a.q_heads; };
    const bool together = (inter || a.rot == 0) && q_vec >= 2 * CP;
    float x[AP_QH][2 * CP];
    if (together) {
#pragma unroll
      for (int h = 0; h < AP_QH; ++h)
        if (has(h)) load_chunk(row + at(h), k, true, q_vec, x[h]);
    } else {
#pragma unroll
      for (int h = 0; h < AP_QH; ++h)
        if (has(h)) load_chunk(row + at(h), k, false, q_vec, x[h]);
    }
    float2 cs[CP];
    if (k.rotated) load_rope(rope + pos * half + k.pair, cs);
#pragma unroll
    for (int h = 0; h < AP_QH; ++h) {
      if (!has(h)) break;
      float y[2 * CP], z[2 * CP];
      from_order(k.rotated && inter, x[h]);
      if (k.rotated) {
        rotate_near(x[h], cs, y);
      } else {
#pragma unroll
        for (int j = 0; j < 2 * CP; ++j) y[j] = x[h][j];
      }
      to_order(y, k.rotated && inter, z);
      if (together) {
        store_n<2 * CP>(out + at(h) + k.a, true, z);
      } else {
        store_n<CP>(out + at(h) + k.a, q_vec >= CP, z);
        store_n<CP>(out + at(h) + k.b, q_vec >= CP, z + CP);
      }
    }
    return;
  }

  const int32_t ph = (int32_t)(block / (uint32_t)units);
  const int32_t u = (int32_t)(block - (uint32_t)ph * (uint32_t)units);
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
  const int rot = is_k ? a.rot : 0, items = m << cpr_log, in_row = (1 << cpr_log) - 1;
  const bool side = is_k && inter, together = (side || rot == 0) && kv_vec >= 2 * CP;

  float y[IT][2 * CP];  // the new elements, first rotated (round_to_odd), then coded
  if (together) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int i = tid + it * AP_T, r = i >> cpr_log;
      if (i < items) load_chunk(rows + r * stride, chunk_of(i & in_row, rot, side), true, kv_vec, y[it]);
    }
  } else {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int i = tid + it * AP_T, r = i >> cpr_log;
      if (i < items) load_chunk(rows + r * stride, chunk_of(i & in_row, rot, side), false, kv_vec, y[it]);
    }
  }
  if (page < 0 || page >= a.b.pages) return;
  uint8_t* codes = (is_k ? a.kc : a.vc) + ((int64_t)page * a.kv_heads + head) * pt * dim;
  float* scale = (is_k ? a.ks : a.vs) + (int64_t)page * a.kv_heads + head;
  const float old = *scale;

  uint32_t top = 0;  // as bits: a NaN is above an infinity, that above every number
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = tid + it * AP_T, r = i >> cpr_log;
    if (i >= items) continue;
    const Chunk k = chunk_of(i & in_row, rot, side);
    if (k.rotated) {
      float2 cs[CP];
      double z[2 * CP];
      from_order(side, y[it]);
      load_rope(rope + (lo + r) * half + k.pair, cs);
      rotate_exact(y[it], cs, z);
#pragma unroll
      for (int j = 0; j < 2 * CP; ++j) y[it][j] = round_to_odd(z[j]);
    }
#pragma unroll
    for (int j = 0; j < 2 * CP; ++j) {
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
    bad = bad || __float_as_uint(old) >= 0x7F800000u;  // negative ones, too
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
  // kernel did not begin) the elements are rotated again and divided in double;
  // so they are where the largest is the largest fp32 number: rotated ones may
  // lie beyond it (the scale is the same up to 1.75 times 2^128, which also is
  // what the codes reach).
  const bool pow2 = (__float_as_uint(now) & 0x7FFFFFu) == 0 && top != 0x7F7FFFFFu;
  const double most = FMT == EFFORT_KV_I8 ? 127.0 : 448.0;
  const float per = (float)(1.0 / (double)now);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = tid + it * AP_T, r = i >> cpr_log;
    if (i >= items) continue;
    const Chunk k = chunk_of(i & in_row, rot, side);
    if (pow2) {
#pragma unroll
      for (int j = 0; j < 2 * CP; ++j) y[it][j] *= per;
    } else if (!bad) {
      float x[2 * CP];
      load_chunk(rows + r * stride, k, false, kv_vec, x);
      from_order(k.rotated && side, x);
      double d[2 * CP];
      if (k.rotated) {
        float2 cs[CP];
        load_rope(rope + (lo + r) * half + k.pair, cs);
        rotate_exact(x, cs, d);
      } else {
#pragma unroll
        for (int j = 0; j < 2 * CP; ++j) d[j] = x[j];
      }
#pragma unroll
      for (int j = 0; j < 2 * CP; ++j)
        y[it][j] = round_to_odd(__builtin_fmin(__builtin_fmax(d[j] / (double)now, -most), most));
    }
    Vec<CP / 4, uint32_t> c[2];
    float z[2 * CP];
    to_order(y[it], k.rotated && side, z);
#pragma unroll
    for (int j = 0; j < CP / 2; ++j)
      c[j / (CP / 4)].e[j % (CP / 4)] =
          bad ? 0u : encode4<FMT>(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
    uint8_t* out = codes + (slot0 + r) * dim;
    typedef Vec<CP / 4, uint32_t> Half;
    if (k.side) {
      *reinterpret_cast<Vec<2, Half>*>(out + k.a) = Vec<2, Half>{{c[0], c[1]}};
    } else {
      *reinterpret_cast<Half*>(out + k.a) = c[0];
      *reinterpret_cast<Half*>(out + k.b) = c[1];
    }
  }
}

template <int DT, int FMT, int IT>
static hipError_t append_it(const AppendArgs& a, hipStream_t s) {
  typedef typename ElemOf<DT>::T T;
  // units: pages that may receive tokens (fewer of the two bounds)
  const int64_t by_page = a.b.tokens / a.page_tokens + 2 * (int64_t)a.b.seqs;
  const int per_token = a.b.tokens <= by_page ? 1 : 0;
  const int64_t units = per_token ? a.b.tokens : by_page;
  const int64_t per_wave = 64 / (a.dim / (2 * CP)) * AP_QH;  // heads
  const int64_t q_waves = (int64_t)a.b.tokens * ((a.q_heads + per_wave - 1) / per_wave);
  const int64_t kv_blocks = units * a.kv_heads * 2, q_blocks = (q_waves + AP_T / 64 - 1) / (AP_T / 64);
  const int64_t blocks = kv_blocks + q_blocks;
  if (blocks > 0x3FFFFFFFll) return hipErrorInvalidValue;  // waves count in 32 bits (2^40 bytes of queries)
  auto vec = [](const void* p, int64_t stride) {
    return rows_aligned<2 * CP, T>(p, stride) ? 2 * CP : rows_aligned<CP, T>(p, stride) ? CP : 1;
  };
  auto less = [](int x, int y) { return x < y ? x : y; };
  const int kv_vec = less(vec(a.k, a.k_stride), vec(a.v, a.v_stride));
  const int q_vec = a.q_heads ? less(vec(a.q, a.q_stride), vec(a.q_out, a.q_out_stride)) : 1;
  // a launch has less than 2^32 threads
  constexpr int64_t most = 0xFFFFFFFFll / AP_T;
  for (int64_t first = 0; first < blocks; first += most) {
    const int64_t n = blocks - first < most ? blocks - first : most;
    hipLaunchKernelGGL((k_append<DT, FMT, IT>), dim3((unsigned)n), dim3(AP_T), 0, s, a, (uint32_t)first,
                       (int32_t)units, per_token, kv_vec, q_vec);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
