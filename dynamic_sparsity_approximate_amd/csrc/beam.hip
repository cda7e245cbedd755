// beam.hip -- beam search's selection: of an item's beams b and their continuations t the
// `keep` best by score[b] + (logit[b][t] - log(sum over t of exp(logit[b][t]))).
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

// Workspace: maxima of groups [rows][groups], then the parts of waves [rows][parts].
struct Part {
  double sum;  // of exp(x - ref_of(top))
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

// NaN-propagating.
__device__ inline float top_of(float x, float y) { return __builtin_elementwise_maximum(x, y); }

template <int CTRL>
__device__ inline float dpp_top(float x) {
  const int b = __float_as_int(x);
  return top_of(x, __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false)));
}

constexpr float kHi = 1.4426950408889634f, kLo = 1.925963033500995e-8f;  // log2(e)
// What a wave's exponentials are relative to: about its largest number, as the power of two
// whose exponent is top * kHi in fp32.  Up to 2^24 that is rounded by 1 or less, and top * kLo
// is below 1, so that the largest's own exponential is between 1/4 and 4 (at -1e10 it would be
// 2^247, infinite).  Larger numbers, -inf and NaN stand for themselves: next to them
// differences that are not exact in fp32 are beyond what an exponential can show.
__device__ inline bool has_power(float top) { return fabsf(top) <= 0x1p24f; }
__device__ inline double ref_of(float top) {
  return has_power(top) ? (double)(top * kHi) * 0.6931471805599453 : (double)top;
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

// A wave works alone: nothing in here waits for another one.  256 rows of 100003 bf16
// logits take 14 us (3.6 TB/s; with waves of 512 logits 18.6); 4 rows of 32000 fp32 ones 3.4,
// a launch and a trip to memory (with waves of 2048 4.2; 64 rows 4.2 and 4.4).  An exponential is two
// products, exact but for 2^-24 of the exponent, whose reference is a number of base 2
// that the sum is kept with, and the instruction's ulp.
template <int DT, int WAVE>
__global__ __launch_bounds__(BM_T) void k_beam_read(BeamArgs a, float* maxima, Part* parts, int64_t first,
                                                    int64_t waves, int64_t per_row, int64_t groups) {
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
    for (int i = 1; i < N; ++i) t = top_of(t, y[it][i]);
    t = dpp_top<0xB1>(t);                    // quad_perm 1032
    t = dpp_top<0x4E>(t);                    // quad_perm 2301
    if (LANES == 8) t = dpp_top<0x141>(t);   // row_half_mirror
    top = top_of(top, t);
    if ((lane & (LANES - 1)) == it % LANES) out = t;
    if (it % LANES == LANES - 1 || it == IT - 1) {  // lane i of a group has the maximum of the i-th of these pieces
      const int my = it - it % LANES + (lane & (LANES - 1));
      const int64_t g = (v0 + (my * 64 + lane) * (int64_t)N) / BM_GROUP;
      if (my <= it && g < groups) maxima[row * groups + g] = out;
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = top_of(top, __shfl_xor(top, d));
  double sum = 0.0;
  if (has_power(top)) {
    const float c = top * kHi;
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      float s[N];
#pragma unroll
      for (int i = 0; i < N; ++i)
        s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(y[it][i], kLo, __builtin_fmaf(y[it][i], kHi, -c)));
#pragma unroll
      for (int d = N / 2; d >= 1; d >>= 1)
#pragma unroll
        for (int i = 0; i < d; ++i) s[i] += s[i + d];
      sum += (double)s[0];
    }
  } else if (top != -INFINITY) {  // (inf - inf is a NaN)
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int i = 0; i < N; ++i) sum += (double)expf(y[it][i] - top);
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
constexpr int BP_RUNS = 2048;  // room for runs
constexpr int BP_FLY = 4;      // maxima of a thread that are on their way together
constexpr int BP_BITS = 14;    // bits of the first bound that are not looked for
static_assert(EFFORT_BEAM_MAX_KEEP * BM_GROUP + EFFORT_BEAM_MAX <= BP_LIST, "the list holds them");
static_assert(EFFORT_BEAM_MAX_KEEP + BP_STEP <= BP_LIST, "the list takes a step more");
static_assert(EFFORT_BEAM_MAX <= 64, "six bits of a beam");

// Calls put(rank, candidate) for each of the list's `n` that has a rank below `keep`; 32
// lanes compare one candidate with the others.
template <typename Put>
__device__ inline void rank_list(const Cand* list, int n, int keep, Put put) {
  const int lane = (int)threadIdx.x & 31, high = (int)threadIdx.x & 32;
  for (int i0 = 0; i0 < n; i0 += BP_T / 32) {
    const int i = i0 + ((int)threadIdx.x >> 5);
    const Cand c = list[i < n ? i : 0];
    int rank = 0;
    for (int j = 0; j < n; j += 32) {
      const uint64_t above = __ballot(j + lane < n && list[j + lane < n ? j + lane : 0] > c);
      rank += __popc((uint32_t)(above >> high));
    }
    if (i < n && rank < keep && lane == 0) put(rank, c);
  }
}

// Bound by its chain of steps: 32 items of 8 beams of 100003 logits, 16 kept, take 9.8 us,
// one of 4 beams of 32000 8.7 (about 3 the sums, 1 each the bound, the runs, the groups and
// the elements); looking at all groups instead of runs first, 20.8 and 9.4.
template <int DT>
__global__ __launch_bounds__(BP_T) void k_beam_pick(BeamArgs a, const float* maxima, const Part* parts, int32_t per_row,
                                                    int32_t groups, int32_t wave_size, int32_t first) {
  typedef typename ElemOf<DT>::T T;
  __shared__ Cand s_list[BP_LIST], s_best[EFFORT_BEAM_MAX_KEEP];
  // log of a beam's sum, and its score (-inf: continues nothing).  They stay apart: next to a
  // large log sum the score would be lost, and the log sum has to meet the logit first.
  __shared__ double s_lse[EFFORT_BEAM_MAX];
  __shared__ float s_near[EFFORT_BEAM_MAX], s_score[EFFORT_BEAM_MAX], s_reach[EFFORT_BEAM_MAX];
  __shared__ uint32_t s_top[BP_T / 4];
  __shared__ int s_n, s_runs;
  __shared__ int32_t s_run[BP_RUNS];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, beams = a.beams, keep = a.keep;
  const int64_t item = (int64_t)first + blockIdx.x, row0 = item * beams;
  auto live = [&](int b) {
    return fabsf(a.scores[row0 + b]) < INFINITY && !(a.ended && a.ended[row0 + b]);
  };

  // a wave for each beam: the sum over its parts
  for (int b = wave; b < beams; b += BP_T / 64) {
    const Part* p = parts + (row0 + b) * per_row;
    const Part mine = p[lane < per_row ? lane : 0];  // on its way with the score
    const bool lives = live(b);
    auto part = [&](int i) { return i < 64 ? mine : p[i]; };
    double ref = -INFINITY, sum = 0.0;
    bool bad = !lives;
    for (int i = lane; lives && i < per_row; i += 64) {
      const Part q = part(i);
      bad = bad || q.sum != q.sum;  // a NaN or an infinity among the logits
      if (q.sum > 0.0 && ref_of(q.top) > ref) ref = ref_of(q.top);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double o = __shfl_xor(ref, d);
      ref = o > ref ? o : ref;
    }
    for (int i = lane; lives && i < per_row; i += 64) {
      const Part q = part(i);
      if (q.sum > 0.0) sum += q.sum * exp(ref_of(q.top) - ref);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    // (0 where all of the row is forbidden)
    const bool some = !__any(bad) && sum > 0.0;
    if (lane == 0) {
      s_lse[b] = some ? ref + log(sum) : 0.0;
      s_near[b] = some ? (float)s_lse[b] : 0.0f;
      s_score[b] = some ? a.scores[row0 + b] : -INFINITY;
    }
  }
  __syncthreads();
  auto value = [&](int b, float x) { return (double)s_score[b] + ((double)x - s_lse[b]); };

  // Runs of neighbouring groups: those of a reading wave, or single groups where there are
  // not many runs for each that is kept.  A first bound, a little too low: of the largest
  // scores that four threads see together, in 32 bits, the keep-th.  Its bits, but for the
  // last ones, are found by one wave.
  const bool coarse = beams * per_row >= 4 * keep;
  const int runs = coarse ? per_row : groups, n = beams * runs;  // at most 2^21
  auto largest = [&](int i) {
    return coarse ? parts[row0 * per_row + i].top : maxima[row0 * groups + i];
  };
  // do(largest, beam, run) for the runs i0 .. i1 - 1; neighbours fall to different fours of threads
  auto each_run = [&](int i0, int i1, auto run) __attribute__((always_inline)) {
    const int own = (tid >> 2) + (tid & 3) * (BP_T / 4);
    int b = (i0 + own) / runs, r = i0 + own - b * runs;
    const int db = BP_T / runs, dr = BP_T % runs;
    for (int i = i0 + own; i < i1; i += BP_FLY * BP_T) {
      float x[BP_FLY];
#pragma unroll
      for (int u = 0; u < BP_FLY; ++u) x[u] = i + u * BP_T < i1 ? largest(i + u * BP_T) : -INFINITY;
#pragma unroll
      for (int u = 0; u < BP_FLY; ++u) {
        if (i + u * BP_T < i1) run(x[u], b, r);
        b += db;
        r += dr;
        if (r >= runs) {
          r -= runs;
          ++b;
        }
      }
    }
  };
  float best = -INFINITY;
  each_run(0, n, [&](float x, int b, int) __attribute__((always_inline)) {
    best = fmaxf(best, (x - s_near[b]) + s_score[b]);
  });
  best = fmaxf(best, __shfl_xor(best, 1));
  best = fmaxf(best, __shfl_xor(best, 2));
  const uint32_t top = order_of(best);
  if ((tid & 3) == 0) s_top[tid >> 2] = top;
  if (tid == 0) s_n = s_runs = 0;
  __syncthreads();
  if (wave == 0) {
    uint32_t mine[BP_T / 256];
#pragma unroll
    for (int u = 0; u < BP_T / 256; ++u) mine[u] = s_top[u * 64 + lane];
    uint32_t least = 0;  // the largest number that `keep` of them reach, two bits at a time
    for (int bit = 30; bit >= BP_BITS; bit -= 2) {
      uint32_t next = least;
#pragma unroll
      for (uint32_t t = 1; t <= 3; ++t) {
        int count = 0;
#pragma unroll
        for (int u = 0; u < BP_T / 256; ++u) count += __popcll(__ballot(mine[u] >= (least | t << bit)));
        if (count >= keep) next = least | t << bit;
      }
      least = next;
    }
    // By beam (a lane each), what a group's maximum has to be: less by more than the
    // roundings, 2^-24 of each of the numbers, of any beam.  A NaN lets nothing pass.
    const bool any = least > order_of(-INFINITY);
    const float bound = fminf(__uint_as_float(least >> 31 ? least & 0x7FFFFFFFu : ~least), 3.0e38f);
    const float near = lane < beams ? s_near[lane] : 0.0f, score = lane < beams ? s_score[lane] : -INFINITY;
    float most = score > -INFINITY ? fmaxf(fabsf(near), fabsf(score)) : 0.0f;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
    const float slack = 0x1p-20f * fabsf(bound) + 0x1p-20f * most;
    const float at = any ? (bound - score - slack) + near : -INFINITY;
    if (lane < beams) s_reach[lane] = score > -INFINITY ? at : __uint_as_float(0x7FC00000u);
  }
  __syncthreads();

  // the groups that reach it, and where they are too many only those that beat the keep-th so far
  Cand bound = {0, 0};
  auto shrink = [&]() __attribute__((always_inline)) {  // to the list's `keep` best, in order
    const int count = s_n;
    rank_list(s_list, count, keep, [&](int rank, const Cand& c) { s_best[rank] = c; });
    __syncthreads();
    const int left = count < keep ? count : keep;
    for (int i = tid; i < left; i += BP_T) s_list[i] = s_best[i];
    if (tid == 0) s_n = left;
    if (left == keep) bound = s_best[keep - 1];
    __syncthreads();
  };
  auto take = [&](float x, int b, int g) __attribute__((always_inline)) {
    if (!(x >= s_reach[b]) || x == -INFINITY) return;
    const Cand c = {order_of(value(b, x)), low_of(b, x, (uint32_t)g)};
    if (!(c > bound)) return;
    const int at = atomicAdd(&s_n, 1);
    if (at < BP_LIST) s_list[at] = c;
  };
  if (coarse) {
    each_run(0, n, [&](float x, int b, int r) __attribute__((always_inline)) {
      if (!(x >= s_reach[b]) || x == -INFINITY) return;
      const int at = atomicAdd(&s_runs, 1);
      if (at < BP_RUNS) s_run[at] = b << 16 | r;
    });
    __syncthreads();
    const int each = wave_size / BM_GROUP, found = s_runs;
    if (found <= BP_RUNS)
      for (int i = tid / each; i < found; i += BP_T / each) {
        const int b = s_run[i] >> 16, g = (s_run[i] & 0xFFFF) * each + tid % each;
        if (g < groups) take(maxima[(row0 + b) * groups + g], b, g);
      }
    __syncthreads();
    if (found > BP_RUNS && tid == 0) s_n = BP_LIST + 1;
  } else {
    each_run(0, n, take);
  }
  __syncthreads();
  if (s_n > BP_LIST) {  // too many alike: step by step
    __syncthreads();
    if (tid == 0) s_n = 0;
    __syncthreads();
    const int all = beams * groups;
    for (int i0 = 0; i0 < all; i0 += BP_STEP) {
      for (int i = i0 + tid; i < i0 + BP_STEP && i < all; i += BP_T)
        take(maxima[row0 * groups + i], i / groups, i % groups);
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
    const Cand c = {order_of(value(b, x)), low_of(b, x, (uint32_t)v)};
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
  const int64_t out = item * keep;
  rank_list(s_list, found, keep, [&](int rank, const Cand& c) {
    const int b = 63 - (int)(c.lo >> 52);
    a.out_scores[out + rank] = (float)number_of(c.hi);
    a.out_parents[out + rank] = (int32_t)(row0 + b);
    const int32_t token = (int32_t)(0xFFFFFu - (uint32_t)(c.lo & 0xFFFFFu));
    a.out_tokens[out + rank] = a.ended && a.ended[row0 + b] ? a.end_token : token;
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
  constexpr int32_t items = 1 << 21;  // of a launch
  for (int32_t first = 0; first < a.items; first += items) {
    const int32_t n = a.items - first < items ? a.items - first : items;
    hipLaunchKernelGGL((k_beam_pick<DT>), dim3((unsigned)n), dim3(BP_T), 0, s, a, maxima, parts, (int32_t)per_row,
                       (int32_t)groups, WAVE, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
static hipError_t beam_dtype(const BeamArgs& a, hipStream_t s) {
  // waves of few logits where larger ones would not fill the chip (figures: k_beam_read)
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
