// beam.hip -- beam search's selection: of an item's beams b and their continuations t the
// `keep` best by score[b] + logit[b][t] - log(sum over t of exp(logit[b][t])).
//
// One pass reads the logits (k_beam_read): a wave has BM_WAVE neighbouring logits of a row
// and leaves their maximum, the sum of their exponentials, and the maximum of every BM_GROUP
// neighbours.  That is enough for k_beam_pick, a block for each item, to name the `keep`
// groups that hold its best: a group that is not among the `keep` best by its largest (ties:
// the lower beam, the larger logit, the lower group) stands behind `keep` groups that each
// hold something better than all it has.  Only these groups are read again.
//
// The order is total: by score in double, then the lower beam, the larger logit, the lower
// token, so that the result does not depend on any order of work.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "host.hpp"
#include "layer.hpp"

namespace effort {

constexpr int BM_GROUP = 32;             // neighbours that share a maximum
constexpr int BM_T = 256;                // threads of a reading block
constexpr int BP_T = 1024;               // of a picking one
constexpr int BM_SMALL = 512, BM_LARGE = 2048;  // logits of a wave, for few rows and for many

// Workspace: maxima of groups [rows][groups], then (maximum, sum) of waves [rows][parts].
struct Part {
  double sum;  // of exp(x - top)
  float top, unused;
};
static int64_t groups_of(int64_t vocab) { return (vocab + BM_GROUP - 1) / BM_GROUP; }
static int64_t parts_of(int64_t vocab, int wave) { return (vocab + wave - 1) / wave; }
static uint64_t maxima_bytes(int64_t rows, int64_t vocab) {
  return ((uint64_t)rows * groups_of(vocab) * sizeof(float) + 255) & ~255ull;
}
uint64_t beam_workspace(int64_t rows, int64_t vocab) {
  return maxima_bytes(rows, vocab) + (uint64_t)rows * parts_of(vocab, BM_SMALL) * sizeof(Part);
}

// ---------------------------------------------------------------- reading

// exp(t) for t <= 0 to about an ulp: t log2(e) as a sum of two floats, the smaller one's
// effect to first order.
__device__ inline float exp_near(float t) {
  const float hi = t * 1.4426950408889634f;
  const float lo = __builtin_fmaf(t, 1.4426950408889634f, -hi) + t * 1.925963033500995e-8f;  // log2(e) beyond fp32
  const float e = __builtin_amdgcn_exp2f(hi);
  return hi < -150.0f ? 0.0f : __builtin_fmaf(e, lo * 0.6931471805599453f, e);  // a NaN stays one
}

template <int CTRL>
__device__ inline float dpp_top(float x) {
  return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(x), __float_as_int(x), CTRL, 0xF, 0xF, false)));
}

// N elements at any address of T's alignment.
template <int N, typename T>
__device__ inline void load_any(const T* p, float* x) {
  struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    T e[N];
  };
  const Loose t = *reinterpret_cast<const Loose*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = (float)t.e[i];
}

// Waits for memory where there are many rows.  A wave works alone: nothing in here waits for
// another one.
template <int DT, int WAVE>
__global__ __launch_bounds__(BM_T) void k_beam_read(BeamArgs a, float* maxima, Part* parts, int64_t first, int64_t waves,
                                                    int64_t per_row, int64_t groups) {
  typedef typename ElemOf<DT>::T T;
  constexpr int N = 16 / sizeof(T), LANES = BM_GROUP / N, IT = WAVE / (64 * N);  // lanes of a group
  const int lane = (int)threadIdx.x & 63;
  const int64_t w = first + (((int64_t)blockIdx.x * BM_T + threadIdx.x) >> 6);
  if (w >= waves) return;
  const int64_t row = w / per_row;
  const int32_t v0 = (int32_t)(w - row * per_row) * WAVE;
  // rows that continue nothing
  const float score = a.scores[row];
  if (!(fabsf(score) < INFINITY) || (a.ended && a.ended[row])) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.stride;
  float y[IT][N];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int32_t v = v0 + (it * 64 + lane) * N;
    if (v + N <= a.vocab) {
      load_any<N>(x + v, y[it]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) y[it][i] = v + i < a.vocab ? (float)x[v + i] : -INFINITY;
    }
  }
  float top = -INFINITY, out = 0.0f;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    float t = y[it][0];
#pragma unroll
    for (int i = 1; i < N; ++i) t = fmaxf(t, y[it][i]);
    t = dpp_top<0xB1>(t);                    // quad_perm 1032
    t = dpp_top<0x4E>(t);                    // quad_perm 2301
    if (LANES == 8) t = dpp_top<0x141>(t);   // row_half_mirror
    top = fmaxf(top, t);
    if ((lane & (LANES - 1)) == it % LANES) out = t;
    if (it % LANES == LANES - 1 || it == IT - 1) {  // lane i of a group has the maximum of the i-th of these pieces
      const int my = it - it % LANES + (lane & (LANES - 1));
      const int64_t g = (v0 + (my * 64 + lane) * (int64_t)N) / BM_GROUP;
      if (my <= it && g < groups) maxima[row * groups + g] = out;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == -INFINITY ? 0.0f : top;
  double sum = 0.0;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = exp_near(y[it][i] - ref);
#pragma unroll
    for (int d = N / 2; d >= 1; d >>= 1)
#pragma unroll
      for (int i = 0; i < d; ++i) s[i] += s[i + d];
    sum += (double)s[0];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) parts[w] = Part{sum, top, 0.0f};
}

// ---------------------------------------------------------------- picking

// A candidate: what comes first in the order is larger.  `hi`: its score; `lo`: the beam
// (6 bits), the logit (32), the group or token (20).
struct Cand {
  uint64_t hi, lo;
};
__device__ inline bool operator>(const Cand& x, const Cand& y) { return x.hi > y.hi || (x.hi == y.hi && x.lo > y.lo); }

// Whole numbers in the order of the numbers.
__device__ inline uint64_t order_of(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ inline double number_of(uint64_t o) { return __builtin_bit_cast(double, o >> 63 ? o & ~(1ull << 63) : ~o); }
__device__ inline uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b >> 31 ? ~b : b | 1u << 31;
}
__device__ inline uint64_t low_of(int beam, float logit, uint32_t at) {
  return (uint64_t)(63 - beam) << 52 | (uint64_t)order_of(logit) << 20 | (0xFFFFFu - at);
}

constexpr int BP_LIST = 4224;  // room of a list: all elements of EFFORT_BEAM_MAX_KEEP groups, and ended beams
constexpr int BP_STEP = 2048;  // groups between two looks at the list's length
static_assert(EFFORT_BEAM_MAX_KEEP * BM_GROUP + EFFORT_BEAM_MAX <= BP_LIST, "the list holds them");
static_assert(EFFORT_BEAM_MAX_KEEP + BP_STEP <= BP_LIST, "the list takes a step more");
static_assert(EFFORT_BEAM_MAX <= 64, "six bits of a beam");

// Calls put(rank, candidate) for each of the list's `n` that has a rank below `keep`.
template <typename Put>
__device__ inline void rank_list(const Cand* list, int n, int keep, Put put) {
  for (int i = (int)threadIdx.x; i < n; i += BP_T) {
    const Cand c = list[i];
    int rank = 0;
    for (int j = 0; j < n && rank < keep; ++j) rank += list[j] > c;
    if (rank < keep) put(rank, c);
  }
}

template <int DT>
__global__ __launch_bounds__(BP_T) void k_beam_pick(BeamArgs a, const float* maxima, const Part* parts, int32_t per_row,
                                                    int32_t groups) {
  typedef typename ElemOf<DT>::T T;
  __shared__ Cand s_list[BP_LIST], s_best[EFFORT_BEAM_MAX_KEEP];
  __shared__ double s_add[EFFORT_BEAM_MAX];  // score minus log of the sum; -inf: continues nothing
  __shared__ uint32_t s_top[BP_T / 4];
  __shared__ uint32_t s_least;
  __shared__ int s_n;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, beams = a.beams, keep = a.keep;
  const int64_t row0 = (int64_t)blockIdx.x * beams;
  auto live = [&](int b) {
    return fabsf(a.scores[row0 + b]) < INFINITY && !(a.ended && a.ended[row0 + b]);
  };

  // a wave for each beam: the sum over its parts
  for (int b = wave; b < beams; b += BP_T / 64) {
    double add = -INFINITY;
    if (live(b)) {
      const Part* p = parts + (row0 + b) * per_row;
      float top = -INFINITY;
      for (int i = lane; i < per_row; i += 64) top = fmaxf(top, p[i].top);
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
      double sum = 0.0;
      for (int i = lane; i < per_row; i += 64) {
        const Part q = p[i];
        sum += q.top == -INFINITY ? q.sum : q.sum * exp((double)q.top - (double)top);
      }
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
      // all of a row forbidden (0), a NaN or an infinity among it (NaN)
      if (sum > 0.0 && top < INFINITY) add = (double)a.scores[row0 + b] - ((double)top + log(sum));
    }
    if (lane == 0) s_add[b] = add;
  }
  __syncthreads();

  const int n = beams * groups;  // at most 2^21
  auto group = [&](int i, Cand* c) {  // whether group i of the item holds a candidate, and its best
    const int b = i / groups, g = i - b * groups;
    const double add = s_add[b];
    if (!(add > -INFINITY)) return false;
    const float x = maxima[(row0 + b) * groups + g];
    if (!(x > -INFINITY)) return false;
    *c = Cand{order_of(add + (double)x), low_of(b, x, (uint32_t)g)};
    return true;
  };
  // A first bound: of the largest scores that four threads see together, rounded to 32
  // bits, the keep-th (rounding keeps the order).  Its bits are found by one wave.
  uint32_t top = 0;
  for (int i = tid; i < n; i += BP_T) {
    Cand c;
    if (!group(i, &c)) continue;
    const uint32_t o = order_of((float)number_of(c.hi));
    top = o > top ? o : top;
  }
  for (int d = 1; d <= 2; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  if ((tid & 3) == 0) s_top[tid >> 2] = top;
  if (tid == 0) s_n = 0;
  __syncthreads();
  if (wave == 0) {
    uint32_t mine[BP_T / 256];
#pragma unroll
    for (int u = 0; u < BP_T / 256; ++u) mine[u] = s_top[u * 64 + lane];
    uint32_t least = 0;  // the largest number that `keep` of them reach
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = least | 1u << bit;
      int count = 0;
#pragma unroll
      for (int u = 0; u < BP_T / 256; ++u) count += __popcll(__ballot(mine[u] >= t));
      if (count >= keep) least = t;
    }
    if (lane == 0) s_least = least;
  }
  __syncthreads();
  const uint32_t least = s_least;

  // the groups that reach it, and as the list fills up only those that beat its keep-th
  Cand bound = {0, 0};
  auto shrink = [&]() {  // to the list's `keep` best, in order
    const int count = s_n;
    rank_list(s_list, count, keep, [&](int rank, const Cand& c) { s_best[rank] = c; });
    __syncthreads();
    const int left = count < keep ? count : keep;
    for (int i = tid; i < left; i += BP_T) s_list[i] = s_best[i];
    if (tid == 0) s_n = left;
    if (left == keep) bound = s_best[keep - 1];
    __syncthreads();
  };
  for (int i0 = 0; i0 < n; i0 += BP_STEP) {
#pragma unroll
    for (int u = 0; u < BP_STEP / BP_T; ++u) {
      const int i = i0 + u * BP_T + tid;
      Cand c;
      if (i < n && group(i, &c) && order_of((float)number_of(c.hi)) >= least && c > bound) s_list[atomicAdd(&s_n, 1)] = c;
    }
    if (i0 + BP_STEP < n) {
      __syncthreads();
      if (s_n > BP_LIST - BP_STEP) shrink();
      __syncthreads();
    }
  }
  __syncthreads();
  shrink();

  // their elements that are at least the last group's largest
  const int count = s_n;
  Cand low = count == keep ? s_best[keep - 1] : Cand{0, 0};
  if (count == keep) low.lo &= ~0xFFFFFull;
  __syncthreads();
  if (tid == 0) s_n = 0;
  __syncthreads();
  for (int i = tid >> 5; i < count; i += BP_T / BM_GROUP) {
    const Cand g = s_best[i];
    const int b = 63 - (int)(g.lo >> 52);
    const int32_t v = (int32_t)(0xFFFFFu - (uint32_t)(g.lo & 0xFFFFFu)) * BM_GROUP + (tid & 31);
    if (v >= a.vocab) continue;
    const float x = (float)static_cast<const T*>(a.logits)[(row0 + b) * a.stride + v];
    const Cand c = {order_of(s_add[b] + (double)x), low_of(b, x, (uint32_t)v)};
    if (x > -INFINITY && (c.hi > low.hi || (c.hi == low.hi && c.lo >= low.lo))) s_list[atomicAdd(&s_n, 1)] = c;
  }
  // an ended beam is its own only continuation
  for (int b = tid; b < beams; b += BP_T) {
    const float s = a.scores[row0 + b];
    if (a.ended && a.ended[row0 + b] && fabsf(s) < INFINITY)
      s_list[atomicAdd(&s_n, 1)] = Cand{order_of((double)s), low_of(b, 0.0f, 0)};
  }
  __syncthreads();
  const int found = s_n;
  const int64_t out = (int64_t)blockIdx.x * keep;
  rank_list(s_list, found, keep, [&](int rank, const Cand& c) {
    const int b = 63 - (int)(c.lo >> 52);
    a.out_scores[out + rank] = (float)number_of(c.hi);
    a.out_parents[out + rank] = (int32_t)(row0 + b);
    a.out_tokens[out + rank] = a.ended && a.ended[row0 + b] ? a.end_token : (int32_t)(0xFFFFFu - (uint32_t)(c.lo & 0xFFFFFu));
  });
  for (int i = found + tid; i < keep; i += BP_T) {
    a.out_scores[out + i] = -INFINITY;
    a.out_parents[out + i] = a.out_tokens[out + i] = -1;
  }
}

// ---------------------------------------------------------------- launches

template <int DT, int WAVE>
static hipError_t beam_wave(const BeamArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.items * a.beams, per_row = parts_of(a.vocab, WAVE), groups = groups_of(a.vocab);
  float* maxima = static_cast<float*>(a.ws);
  Part* parts = reinterpret_cast<Part*>(static_cast<char*>(a.ws) + maxima_bytes(rows, a.vocab));
  constexpr int64_t most = 0xFFFFFFFFll / BM_T;  // a launch has less than 2^32 threads
  const int64_t waves = rows * per_row;
  for (int64_t first = 0; first < waves; first += most * (BM_T / 64)) {
    const int64_t blocks = (waves - first + BM_T / 64 - 1) / (BM_T / 64);
    hipLaunchKernelGGL((k_beam_read<DT, WAVE>), dim3((unsigned)(blocks < most ? blocks : most)), dim3(BM_T), 0, s, a,
                       maxima, parts, first, waves, per_row, groups);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_beam_pick<DT>), dim3((unsigned)a.items), dim3(BP_T), 0, s, a, maxima, parts, (int32_t)per_row,
                     (int32_t)groups);
  return hipGetLastError();
}

template <int DT>
static hipError_t beam_dtype(const BeamArgs& a, hipStream_t s) {
  // waves of few logits where larger ones would not fill the chip
  const int64_t waves = (int64_t)a.items * a.beams * parts_of(a.vocab, BM_LARGE);
  return waves < 8 * (int64_t)cu_count() ? beam_wave<DT, BM_SMALL>(a, s) : beam_wave<DT, BM_LARGE>(a, s);
}

hipError_t launch_beam(const BeamArgs& a, int32_t dtype, hipStream_t s) {
  switch (dtype) {
    case EFFORT_F32: return beam_dtype<EFFORT_F32>(a, s);
    case EFFORT_F16: return beam_dtype<EFFORT_F16>(a, s);
    case EFFORT_BF16: return beam_dtype<EFFORT_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace effort
