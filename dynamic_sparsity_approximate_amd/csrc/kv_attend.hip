// kv_attend.hip -- causal attention over the paged 8-bit cache.
//
// For one sequence and one head of the cache, the rows of the products are the
// (new token, query head of the group) pairs, token by token: row = token *
// group + query head.  A wave multiplies 16 rows with 32 tokens at a time:
//   S^T[token][row] = K Q^T, two 16x16x32 products per 32 elements of a head,
//   O^T[element][row] += V^T P^T, one product per 16 elements of a head.
// In S^T a lane holds its row (lane mod 16) at tokens (lane / 16) * 4 + 0..3 of
// both 16-token halves: exactly the eight tokens that it has to supply of P^T
// when the second product counts its tokens in that order, so the weights never
// leave their lane, and a row's maximum, sum and rescaling are the lane's own
// but for two exchanges across the four lanes of a row.
// Codes become fp16 exactly (8 bits fit its 11); q is scaled per row by a power
// of two into fp16's upper range.  fp32 rows of q, and the weights, are taken as
// two fp16 parts each (22 bits) and the products run twice.  Only prompts with
// 16-bit rows take the weights' upper part alone (11 bits, fewer below 2^-20 of
// the reference): the other costs k_attend_split, which waits for memory, 0.2 to
// 3 per cent, but two bf16 prompts of 4096 tokens 426 us instead of 317, for
// errors of 2.07e-4 instead of 2.7e-4 (fp16) or 1.65e-3 instead of 1.66e-3 (bf16)
// of the outputs, most of which is their own last rounding.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "host.hpp"
#include "layer.hpp"

namespace effort {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int AT_T = 256, AT_W = AT_T / 64;
constexpr int AT_TILE = 32;              // tokens of one step of a wave
constexpr int AT_CHUNK = AT_W * AT_TILE; // tokens of one step of a block
constexpr float kLog2e = 1.4426950408889634f;
// Weights are held times 2^6 relative to a row's reference score, which follows
// the row's maximum only when that is 2^8 times larger (most steps then rescale
// nothing), and the unit of values (below) may double them: at most 2^15, inside
// fp16, whose normal numbers begin 2^-20 below the reference.
constexpr float kWeightExp = 6.0f, kSlack = 8.0f;

// ---------------------------------------------------------------- pieces of both products

// NaN-propagating (and one instruction, for three operands too).
__device__ inline float max_of(float x, float y) { return __builtin_elementwise_maximum(x, y); }

__device__ inline float max_of_row(float x) {  // over the four lanes that share a row
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = max_of(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_of(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ inline float sum_of_row(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int CTRL>
__device__ inline float dpp_max(float x) {
  return max_of(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true)));
}
// Over four neighbouring lanes.
__device__ inline float quad_max(float x) { return dpp_max<0x4E>(dpp_max<0xB1>(x)); }  // quad_perm 1032, 2301

__device__ inline float lane_of(float x, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}
__device__ inline float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }

// Two codes (bytes 0, 1 or 2, 3 of w) as fp16, exactly.
template <int FMT, bool HI>
__device__ inline h2 decode2(uint32_t w) {
  if (FMT == EFFORT_KV_I8) {
    // code + 128 in the low bits of the fp16 number 1024 + (code + 128)
    const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w ^ 0x80808080u, HI ? 0x07030602u : 0x05010400u);
    const h2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(h2, u) - bias;
  }
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
}

__device__ inline h8 join8(h2 a, h2 b, h2 c, h2 d) {
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int FMT>
__device__ inline h8 decode8(uint32_t lo, uint32_t hi) {
  return join8(decode2<FMT, false>(lo), decode2<FMT, true>(lo), decode2<FMT, false>(hi), decode2<FMT, true>(hi));
}

// Eight weights as fp16, and what that leaves off as fp16 too.
__device__ inline h8 weights8(const float* p) {
  h8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (_Float16)p[i];
  return r;
}

__device__ inline h8 rest8(const float* p, h8 w) {
  h8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (_Float16)(p[i] - (float)w[i]);
  return r;
}

// The power of two that brings a row whose largest magnitude is `top` to [2^13, 2^14).
__device__ inline float power_of_row(float top) {
  int up = 13 - ((int)(__float_as_uint(top) >> 23) - 127);
  up = top > 0.0f && top < INFINITY ? (up > 100 ? 100 : up) : 0;
  return __uint_as_float((uint32_t)(up + 127) << 23);
}

// What the products of a row scaled so, with codes, are multiplied by to be scores
// in base 2, but for a key's scale: NaN for a row with an infinity, whose products
// alone could all be -inf, as if the row saw nothing.
__device__ inline float factor_of_row(float scale, float top, float by) {
  return top < INFINITY ? fabsf(scale) * kLog2e / by : __uint_as_float(0x7FC00000u);
}

// The tokens after `low`, up to `high`, that a row at `pos` sees of `to` tokens.
struct Sight {
  int32_t low, high;
};
__device__ inline Sight sight_of(int64_t pos, int32_t to, int32_t window) {
  Sight v;
  v.high = pos < to ? (int32_t)(pos < -1 ? -1 : pos) : to - 1;
  v.low = window && pos - window > -1 ? (int32_t)(pos - window < to ? pos - window : to) : -1;
  return v;
}

// ---------------------------------------------------------------- who does what

// A sequence's part of a call.
struct Seq {
  int32_t first, n;   // its rows of q
  int64_t pos;        // position of its first new token
  int32_t lo, hi;     // tokens that any row sees, lo a multiple of AT_TILE
  int32_t tiles;      // row tiles of `rows` rows
  int32_t chunks;     // of AT_CHUNK tokens
};

__device__ inline Seq seq_of(const AttendArgs& a, int s, int group, int rows) {
  Seq q;
  const int32_t s0 = start_of(a.b, s), s1 = start_of(a.b, s + 1);
  q.first = s0;
  q.n = s1 > s0 ? s1 - s0 : 0;
  const int64_t len = a.b.lens[s], cap = (int64_t)a.b.max_pages * a.page_tokens;
  q.pos = len - q.n;
  const int64_t from = a.window && q.pos + 1 > a.window ? q.pos + 1 - a.window : 0;
  const int64_t to = len < cap ? len : cap;
  q.tiles = (int32_t)(((int64_t)q.n * group + rows - 1) / rows);
  q.chunks = 0;
  q.lo = q.hi = 0;
  if (q.n > 0 && to > from) {
    q.lo = (int32_t)(from & ~(int64_t)(AT_TILE - 1));
    q.hi = (int32_t)to;
    q.chunks = (int32_t)((to - q.lo + AT_CHUNK - 1) / AT_CHUNK);
  }
  return q;
}

__device__ inline uint64_t chunks_of(const AttendArgs& a, int s, int group, int rows) {
  const Seq q = seq_of(a, s, group, rows);
  return (uint64_t)q.tiles * (uint64_t)a.kv_heads * (uint64_t)q.chunks;
}

// Chunks before the sequences, one entry for `per` of them (one each up to 256
// sequences); every block computes it from the lengths, so that a captured call
// follows them.
struct Plan {
  uint64_t before[AT_T + 1];
  uint64_t part[AT_W];
};
__device__ inline int per_entry(const AttendArgs& a) { return (a.b.seqs + AT_T - 1) / AT_T; }

// Returns all sequences' chunks; for one sequence that is all there is to know.
__device__ uint64_t make_plan(const AttendArgs& a, int group, int rows, Plan* p) {
  if (a.b.seqs == 1) return chunks_of(a, 0, group, rows);
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6, per = per_entry(a);
  uint64_t sum = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < a.b.seqs) sum += chunks_of(a, tid * per + i, group, rows);
  uint64_t run = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) p->part[wave] = run;
  __syncthreads();
  uint64_t base = run - sum;
  for (int w = 0; w < wave; ++w) base += p->part[w];
  p->before[tid] = base;
  if (tid == AT_T - 1) p->before[AT_T] = base + sum;
  __syncthreads();
  return p->before[AT_T];
}

// Chunks before sequence s.
__device__ inline uint64_t start_of_seq(const AttendArgs& a, const Plan& p, int s, int group, int rows) {
  if (a.b.seqs == 1) return 0;
  const int per = per_entry(a);
  uint64_t c = p.before[s / per];
  for (int i = s / per * per; i < s; ++i) c += chunks_of(a, i, group, rows);
  return c;
}

// The sequence that owns chunk c (of those that have chunks), at or after `from`.
__device__ inline int owner(const AttendArgs& a, const Plan& p, uint64_t c, int group, int rows) {
  if (a.b.seqs == 1) return 0;
  const int per = per_entry(a);
  int lo = 0, hi = AT_T;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.before[mid] <= c) lo = mid; else hi = mid;
  }
  int s = lo * per;
  uint64_t at = p.before[lo];
  for (;;) {
    const uint64_t n = chunks_of(a, s, group, rows);
    if (c < at + n || s + 1 >= a.b.seqs) return s;
    at += n;
    ++s;
  }
}

// ---------------------------------------------------------------- split over blocks

// A wave takes 32 tokens at a time; its keys' codes are asked for again as soon
// as the scores are done with them, its values' as soon as the weighted sum is:
// each is on its way during the other's work, with one set of registers.
//
// Blocks share the (sequence, head, row tile) items' chunks evenly, in order:
// block b takes the chunks [b W / B, (b + 1) W / B) of all W (B: the grid, or W
// if that is less).  An item that one block has whole is finished there; the
// others leave (maximum, sum, weighted values) of their part for k_attend_join.
// A decode batch of unequal lengths keeps every CU busy to the end without the
// host knowing the lengths.  With WHOLE a block takes one item to its end, for
// tables of so few tokens that joining would cost more than it saves.
// Bound by memory once there are some ten chunks for each block: 64 sequences of
// 4000 to 16384 int8 tokens are read at 5.2 TB/s, one of 200003 e4m3 tokens at
// 5.0, 16 of 1000 to 8192 at 4.1 (with the join 3.6).
// `RT`: 16-row tiles of an item, `NW`: waves of a block.
template <int DT, int FMT, int D, int RT, int NW, bool WHOLE>
__global__ __launch_bounds__(64 * NW, 2) void k_attend_split(AttendArgs a, float* parts) {
  typedef typename ElemOf<DT>::T T;
  constexpr bool SPLIT = DT == EFFORT_F32;
  constexpr int KS = D / 32, ND = D / 16, ROWS = 16 * RT, LD = D + 4, THREADS = 64 * NW, STEP = NW * AT_TILE;
  static_assert(WHOLE || NW == AT_W, "a chunk is a step of a block");
  __shared__ Plan s_plan;
  __shared__ float s_o[NW][ROWS][LD];
  __shared__ float s_m[NW][ROWS], s_l[NW][ROWS], s_u[NW];
  __shared__ int s_seq;
  const int tid = (int)threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.q_heads / a.kv_heads, shift = __builtin_ctz(a.page_tokens), in_page = (1 << shift) - 1;
  uint64_t c = 0, c_end = 1;
  int s = 0;
  if (WHOLE) {
    auto base = [&](int i) { return (int64_t)start_of(a.b, i) * group / ROWS + i; };
    if (a.b.seqs > 1) {
      if (tid == 0) s_seq = a.b.seqs;
      __syncthreads();
      for (int i = tid; i < a.b.seqs; i += THREADS)
        if (base(i) <= blockIdx.y && blockIdx.y < base(i + 1)) atomicMin(&s_seq, i);
      __syncthreads();
      s = __builtin_amdgcn_readfirstlane(s_seq);
      if (s >= a.b.seqs) return;
    }
  } else {
    const uint64_t total = make_plan(a, group, ROWS, &s_plan);
    const uint64_t nb = total < gridDim.x ? total : gridDim.x;  // no block has nothing
    if (blockIdx.x >= nb) return;
    c = total * blockIdx.x / nb;
    c_end = total * (blockIdx.x + 1) / nb;
    s = __builtin_amdgcn_readfirstlane(owner(a, s_plan, c, group, ROWS));
  }
  uint64_t s_start = WHOLE ? 0 : start_of_seq(a, s_plan, s, group, ROWS);
  while (c < c_end) {
    const Seq q = seq_of(a, s, group, ROWS);
    int head, tile;
    uint32_t ch0 = 0, take = 1;
    if (WHOLE) {
      head = (int)blockIdx.x;
      tile = (int)(blockIdx.y - ((int64_t)q.first * group / ROWS + s));
      if (tile < 0 || tile >= q.tiles) return;
      take = (uint32_t)q.chunks;
    } else {
      const uint64_t mine = (uint64_t)q.tiles * (uint64_t)a.kv_heads * (uint64_t)q.chunks;
      if (c >= s_start + mine) {
        s_start += mine;
        if (++s >= a.b.seqs) return;
        continue;
      }
      const uint64_t in = c - s_start;
      const uint32_t item = (uint32_t)(in / (uint32_t)q.chunks);
      ch0 = (uint32_t)(in % (uint32_t)q.chunks);
      head = (int)(item / (uint32_t)q.tiles);
      tile = (int)(item % (uint32_t)q.tiles);
      const uint32_t left = q.chunks - ch0;
      take = c_end - c < left ? (uint32_t)(c_end - c) : left;
    }
    const bool whole = WHOLE || (ch0 == 0 && take == (uint32_t)q.chunks);
    const int32_t* table = a.b.table + s * a.b.table_stride;
    const int rows = q.n * group - tile * ROWS < ROWS ? q.n * group - tile * ROWS : ROWS;
    const int32_t t_begin = q.lo + (int32_t)(ch0 * AT_CHUNK) + wave * AT_TILE;
    const int64_t stop = (int64_t)q.lo + (int64_t)(ch0 + take) * AT_CHUNK;
    const int32_t t_end = stop < q.hi ? (int32_t)stop : q.hi;

    // pages of the two 16-token halves of the step at t; -1: none, or not this block's
    struct Two {
      int32_t p[2];
    };
    auto pages_at = [&](int32_t t) {
      Two r;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        r.p[u] = t < t_end && t + 16 * u < q.hi ? table[(t + 16 * u) >> shift] : -1;
        r.p[u] = __builtin_amdgcn_readfirstlane(r.p[u]);
      }
      return r;
    };
    auto there = [&](int32_t p) { return p >= 0 && p < a.b.pages; };
    auto head_at = [&](int32_t p) { return (int64_t)(there(p) ? p : 0) * a.kv_heads + head; };  // page 0: never used
    uint4 kc[2][D / 64];
    uint32_t vc[2][4][D / 64];
    float ks[2], vs[2];
    auto load_keys = [&](int32_t t, const Two& pg) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t ph = head_at(pg.p[u]);
        const uint8_t* from = a.kc + ((ph << shift) + ((t + 16 * u) & in_page)) * D + (j * D + g * 16);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) kc[u][x] = *reinterpret_cast<const uint4*>(from + 64 * x);
        ks[u] = a.ks[ph];
      }
    };
    auto load_values = [&](int32_t t, const Two& pg) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t ph = head_at(pg.p[u]);
        const uint8_t* from = a.vc + ((ph << shift) + ((t + 16 * u) & in_page)) * D + (g * 4 * D + j * (D / 16));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2*>(from + r * D);
            vc[u][r][0] = w.x;
            vc[u][r][D / 64 - 1] = w.y;
          } else {
            vc[u][r][0] = *reinterpret_cast<const uint32_t*>(from + r * D);
          }
        }
        vs[u] = a.vs[ph];
      }
    };
    Two now = pages_at(t_begin), next = pages_at(t_begin + STEP);
    load_keys(t_begin, now);
    load_values(t_begin, now);

    // the rows' queries, scaled by a power of two to at most 2^14; the sign of
    // the call's scale goes into them
    h8 qh[RT][KS], ql[RT][KS];
    float f[RT];
    Sight see[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      int r = rt * 16 + j;
      r = tile * ROWS + (r < rows ? r : rows - 1);  // rows behind the last one repeat it
      const int i = r / group;
      see[rt] = sight_of(q.pos + i, q.hi, a.window);
      const T* src = static_cast<const T*>(a.q) + (q.first + i) * a.q_stride +
                     (int64_t)(head * group + r - i * group) * D + g * 16;
      float x[KS][8], top = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) load_n<8>(src + (k >> 1) * 64 + (k & 1) * 8, a.q_vec != 0, x[k]);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[k][e]));
      top = max_of_row(top);
      const float by = power_of_row(top);
      f[rt] = factor_of_row(a.scale, top, by);
      const float mul = a.scale < 0.0f ? -by : by;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= mul;
        qh[rt][k] = weights8(x[k]);
        if (SPLIT) ql[rt][k] = rest8(x[k], qh[rt][k]);
      }
    }
    const int32_t row0 = tile * ROWS, row1 = row0 + rows - 1;
    const Sight see0 = sight_of(q.pos + row0 / group, q.hi, a.window);  // of the first row and the last
    const Sight see1 = sight_of(q.pos + row1 / group, q.hi, a.window);

    f4 o[RT][ND];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = -INFINITY;
      l[rt] = 0.0f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[rt][d] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // O counts in `unit`s of the values' scale: a token of scale vs weighs w * vs /
    // unit.  The unit follows the scales up at once, down when they are 2^10
    // smaller (but never to where what is there could overflow).
    float unit = 0.0f, per_unit = 0.0f, unit_top = 0.0f;

    for (int32_t t = t_begin; t < t_end; t += STEP) {
      // a half that no row sees counts as absent: its page may have any scale
      const bool ok0 = there(now.p[0]) && t + 15 > see0.low && t <= see1.high;
      const bool ok1 = there(now.p[1]) && t + 31 > see0.low && t + 16 <= see1.high;
      f4 sc[RT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint4 w = kc[u][k >> 1];
          const h8 kf = (k & 1) ? decode8<FMT>(w.z, w.w) : decode8<FMT>(w.x, w.y);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            sc[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qh[rt][k], sc[rt][u], 0, 0, 0);
            if (SPLIT) sc[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, ql[rt][k], sc[rt][u], 0, 0, 0);
          }
        }
      }
      // a poisoned page: its scores are NaN, its values count as any
      const bool bad0 = __float_as_uint(ks[0]) >= 0x7F800000u || __float_as_uint(vs[0]) >= 0x7F800000u;
      const bool bad1 = __float_as_uint(ks[1]) >= 0x7F800000u || __float_as_uint(vs[1]) >= 0x7F800000u;
      const float k0 = bad0 ? __uint_as_float(0x7FC00000u) : ks[0], k1 = bad1 ? __uint_as_float(0x7FC00000u) : ks[1];
      load_keys(t + STEP, next);
      float w[RT][8];
      const bool full = ok0 && ok1 && t + AT_TILE - 1 <= see0.high && t > see1.low;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float c0 = f[rt] * k0, c1 = f[rt] * k1;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[rt][i] = sc[rt][i >> 2][i & 3] * (i < 4 ? c0 : c1);
        if (!full) {
          const int32_t low = see[rt].low - t - g * 4, high = see[rt].high - t - g * 4;
          const int32_t high0 = ok0 ? high : -AT_TILE, high1 = ok1 ? high : -AT_TILE;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (i >> 2) * 16 + (i & 3);
            if (at > (i < 4 ? high0 : high1) || at <= low) w[rt][i] = -INFINITY;
          }
        }
        float top = w[rt][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = max_of(top, w[rt][i]);
        top = max_of_row(top);
        if (__any(top > m[rt] + kSlack)) {
          const float mn = fmaxf(top, m[rt]);
          const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
          m[rt] = mn;
          l[rt] *= alpha;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[rt][d] *= alpha;
        }
        // nothing seen so far (or only NaN): the weights are 0 (or NaN)
        const float ref = (m[rt] == -INFINITY ? 0.0f : m[rt]) - kWeightExp;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[rt][i] = __builtin_amdgcn_exp2f(w[rt][i] - ref);
        l[rt] += ((w[rt][0] + w[rt][1]) + (w[rt][2] + w[rt][3])) + ((w[rt][4] + w[rt][5]) + (w[rt][6] + w[rt][7]));
      }
      if (!full) {  // values of tokens that no row sees weigh 0, so they must not be NaN
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!(u ? ok1 : ok0) || t + 16 * u + g * 4 + r >= q.hi || t + 16 * u + g * 4 + r <= see0.low) {
#pragma unroll
              for (int x = 0; x < D / 64; ++x) vc[u][r][x] = 0u;
            }
      }
      // Halves whose scales are far apart are weighed one after the other: the
      // smaller's weights would lose bits below the larger's.
      const float v0 = ok0 && !bad0 ? vs[0] : 0.0f, v1 = ok1 && !bad1 ? vs[1] : 0.0f;
      const bool apart = fminf(v0, v1) > 0.0f && fmaxf(v0, v1) > 0x1p10f * fminf(v0, v1);
#pragma unroll 1
      for (int pass = 0; pass < (apart ? 2 : 1); ++pass) {
        const float s0 = pass == 0 ? v0 : 0.0f, s1 = apart && pass == 0 ? 0.0f : v1, top = fmaxf(s0, s1);
        unit_top = fmaxf(unit_top, top);
        if (top > 2.0f * unit || (top < 0x1p-10f * unit && top > 0.0f)) {
          const float to = fmaxf(fmaxf(top, unit_top * 0x1p-60f), 0x1p-100f), by = unit / to;
          unit = to;
          per_unit = 1.0f / to;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[rt][d] *= by;
        }
        const float rel0 = bad0 && pass == 0 ? 1.0f : s0 * per_unit, rel1 = bad1 && pass == 0 ? 1.0f : s1 * per_unit;
        h8 ph[RT], pl[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = w[rt][i] * (i < 4 ? rel0 : rel1);
          ph[rt] = weights8(y);
          pl[rt] = rest8(y, ph[rt]);
        }
        // weighted values: element n * ND + d of a head is row n of product d
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          uint32_t e[4], e2[4];  // both tokens of a pair: bytes 0 and 1, bytes 2 and 3
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t lo = vc[h >> 1][(h & 1) * 2][x], hi = vc[h >> 1][(h & 1) * 2 + 1][x];
            e[h] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
            e2[h] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
          }
          const h8 vf[4] = {join8(decode2<FMT, false>(e[0]), decode2<FMT, false>(e[1]), decode2<FMT, false>(e[2]),
                                  decode2<FMT, false>(e[3])),
                            join8(decode2<FMT, true>(e[0]), decode2<FMT, true>(e[1]), decode2<FMT, true>(e[2]),
                                  decode2<FMT, true>(e[3])),
                            join8(decode2<FMT, false>(e2[0]), decode2<FMT, false>(e2[1]), decode2<FMT, false>(e2[2]),
                                  decode2<FMT, false>(e2[3])),
                            join8(decode2<FMT, true>(e2[0]), decode2<FMT, true>(e2[1]), decode2<FMT, true>(e2[2]),
                                  decode2<FMT, true>(e2[3]))};
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              f4& acc = o[rt][x * 4 + d];
              acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], ph[rt], acc, 0, 0, 0);
              acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[d], pl[rt], acc, 0, 0, 0);
            }
        }
      }
      load_values(t + STEP, next);
      now = next;
      next = pages_at(t + 2 * STEP);
    }

    // the waves' parts become one
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float lt = sum_of_row(l[rt]);
      if (g == 0) {
        s_m[wave][rt * 16 + j] = m[rt];
        s_l[wave][rt * 16 + j] = lt;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int x = 0; x < ND / 4; ++x)
          *reinterpret_cast<f4*>(&s_o[wave][rt * 16 + j][(g * 4 + r) * ND + x * 4]) =
              f4{o[rt][x * 4][r], o[rt][x * 4 + 1][r], o[rt][x * 4 + 2][r], o[rt][x * 4 + 3][r]};
    }
    if (lane == 0) s_u[wave] = unit;
    __syncthreads();
    // slot 0: a part that does not start its item, slot 1: one that does
    float* mine = parts + ((int64_t)blockIdx.x * 2 + (ch0 == 0 ? 1 : 0)) * ROWS * (D + 2);
    for (int i = tid; i < rows * (D / 4); i += THREADS) {
      const int r = i / (D / 4), x = (i % (D / 4)) * 4;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w][r]);
      const float ref = top == -INFINITY ? 0.0f : top;
      f4 v = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float e = __builtin_amdgcn_exp2f(s_m[w][r] - ref);
        // a wave that saw only NaN has no maximum: its sum stays NaN
        sum += s_m[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * e;
        v += *reinterpret_cast<const f4*>(&s_o[w][r][x]) * (e * s_u[w]);
      }
      if (whole) {
        const int row = tile * ROWS + r, tok = row / group;
        T* out = static_cast<T*>(a.out) + (q.first + tok) * a.out_stride +
                 (int64_t)(head * group + row - tok * group) * D + x;
        const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = (T)(v[k] * by);
      } else {
        *reinterpret_cast<f4*>(mine + r * D + x) = v;
        if (x == 0) {
          mine[ROWS * D + r] = top;
          mine[ROWS * D + ROWS + r] = sum;
        }
      }
    }
    if (WHOLE) return;
    c += take;
  }
}

// Joins `count` parts of a row by 256 / R threads: a group of 32 has D / 32
// elements each of every (8 / R)-th part, four parts in flight, with the
// maximum and sum of what it has seen; then the groups are joined the same way.
// `at(i)` is part i: the values of `rows` rows, their maxima, their sums.
template <int D, int R, typename T, typename At>
__device__ void join_row(int count, int rows, int r, At at, T* out) {
  constexpr int E = D / 32, GROUPS = 8 / R, FLY = 4;
  __shared__ float s_m[8], s_l[8];
  __shared__ float s_v[8][D];
  const int tid = (int)threadIdx.x, lane = tid & 31, slot = tid >> 5, k = slot % GROUPS;
  float m = -INFINITY, l = 0.0f, v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.0f;
  for (int i0 = k; i0 < count; i0 += GROUPS * FLY) {
    float mi[FLY], li[FLY];
    Vec<E, float> y[FLY];
#pragma unroll
    for (int j = 0; j < FLY; ++j) {
      const int i = i0 + j * GROUPS;
      const float* p = at(i < count ? i : i0);
      mi[j] = i < count ? p[rows * D + r] : -INFINITY;
      li[j] = i < count ? p[rows * D + rows + r] : 0.0f;
      y[j] = *reinterpret_cast<const Vec<E, float>*>(p + r * D + lane * E);
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < FLY; ++j) top = fmaxf(top, mi[j]);
    const float ref = top == -INFINITY ? 0.0f : top, was = __builtin_amdgcn_exp2f(m - ref);
    // a part that saw only NaN has no maximum: its sum stays NaN
    l = m == -INFINITY ? l : l * was;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= was;
    m = top;
#pragma unroll
    for (int j = 0; j < FLY; ++j) {
      const float by = __builtin_amdgcn_exp2f(mi[j] - ref);
      l += mi[j] == -INFINITY ? li[j] : li[j] * by;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = by > 0.0f ? __builtin_fmaf(y[j].e[e], by, v[e]) : v[e];
    }
  }
  if (GROUPS > 1) {
    if (lane == 0) {
      s_m[slot] = m;
      s_l[slot] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_v[slot][lane * E + e] = v[e];
    __syncthreads();
    if (k != 0) return;
    float top = m;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) top = fmaxf(top, s_m[slot + g]);
    const float ref = top == -INFINITY ? 0.0f : top, was = __builtin_amdgcn_exp2f(m - ref);
    l = m == -INFINITY ? l : l * was;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= was;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const float mg = s_m[slot + g], by = __builtin_amdgcn_exp2f(mg - ref);
      l += mg == -INFINITY ? s_l[slot + g] : s_l[slot + g] * by;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = __builtin_fmaf(s_v[slot + g][lane * E + e], by, v[e]);
    }
  }
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = (T)(v[e] * by);
}

// Joins the parts that blocks left of an item, and writes the rows that see
// nothing.  One block per (R rows, head); row tiles of a sequence are counted
// from first * group / ROWS + s, enough for every sequence before it.
template <int DT, int D, int RT, int R>
__global__ __launch_bounds__(AT_T) void k_attend_join(AttendArgs a, const float* parts, uint32_t nb32) {
  typedef typename ElemOf<DT>::T T;
  constexpr int ROWS = 16 * RT;
  __shared__ Plan s_plan;
  __shared__ int s_seq;
  const int tid = (int)threadIdx.x, head = (int)blockIdx.y, group = a.q_heads / a.kv_heads;
  const uint32_t bt = blockIdx.x / (ROWS / R);
  const int r0 = (int)(blockIdx.x % (ROWS / R)) * R;
  auto base = [&](int i) { return (int64_t)start_of(a.b, i) * group / ROWS + i; };
  int s = 0;
  if (a.b.seqs > 1) {
    if (tid == 0) s_seq = a.b.seqs;
    __syncthreads();
    for (int i = tid; i < a.b.seqs; i += AT_T)
      if (base(i) <= bt && bt < base(i + 1)) atomicMin(&s_seq, i);
    __syncthreads();
    s = s_seq;
    if (s >= a.b.seqs) return;
  }
  const Seq q = seq_of(a, s, group, ROWS);
  const int64_t at_tile = (int64_t)bt - base(s);
  if (at_tile < 0 || at_tile * ROWS + r0 >= (int64_t)q.n * group) return;
  const int tile = (int)at_tile;
  const int r = r0 + (tid >> 5) / (8 / R);
  const bool mine = tile * ROWS + r < q.n * group;
  const int row = mine ? tile * ROWS + r : tile * ROWS + r0, tok = row / group;
  T* out = static_cast<T*>(a.out) + (q.first + tok) * a.out_stride + (int64_t)(head * group + row - tok * group) * D;
  if (q.chunks == 0) {
    for (int i = tid & 31; i < D; i += 32) out[i] = (T)0.0f;
    return;
  }
  const uint64_t total = make_plan(a, group, ROWS, &s_plan), nb = total < nb32 ? total : nb32;
  const uint64_t c0 = start_of_seq(a, s_plan, s, group, ROWS) +
                      ((uint64_t)head * q.tiles + tile) * q.chunks;
  const uint64_t c1 = c0 + q.chunks - 1;
  const uint64_t b0 = ((c0 + 1) * nb - 1) / total, b1 = ((c1 + 1) * nb - 1) / total;  // blocks of its first, last chunk
  if (b0 == b1) return;
  const float* first = parts + (b0 * 2 + 1) * (uint64_t)(ROWS * (D + 2));
  const float* rest = parts + (b0 + 1) * 2 * (uint64_t)(ROWS * (D + 2));
  auto at = [&](int i) { return i == 0 ? first : rest + (uint64_t)(i - 1) * 2 * (ROWS * (D + 2)); };
  // a row behind the last one repeats the block's first
  join_row<D, R>((int)(b1 - b0) + 1, ROWS, mine ? r : r0, at, out);
}

// ---------------------------------------------------------------- prompts

// Rows of a block: RT 16-row tiles a wave.  Two for prompts that fill the chip;
// one for shorter ones (prompt_shape), for twice the blocks and (heads of 64
// elements) three of them on a CU.
template <int RT>
constexpr int prompt_rows() {
  return 16 * RT * AT_W;
}
constexpr int PR_TILE = 64;         // tokens of one step
constexpr int PR_SUB = PR_TILE / 16;

// 16-byte pieces of a step in LDS, as fp16: keys [token][piece of 8 elements],
// values [element, in the products' order][piece of 8 tokens, in the order in
// which the product of weights and values counts them].  The pieces of a row
// are exchanged so that 16 neighbouring lanes' accesses, reading and writing,
// fall on 16 different pieces of 256 bytes.
template <int D>
__device__ inline int key_piece(int token, int piece) {
  return D == 128 ? token * 16 + (piece ^ (token & 15)) : token * 8 + (piece ^ (token >> 1 & 7));
}
template <int D>
__device__ inline int value_piece(int element, int piece) {
  constexpr int ND = D / 16;
  const int d = element % ND, j = element / ND;
  return (d * 16 + j) * (PR_TILE / 8) + (piece ^ (j >> 1 & 7) ^ (d >> 2 << 2));
}

// What a thread carries of a step from memory to LDS: D / 64 times 16 codes of a
// key, and 4 elements of 8 tokens' values.
template <int D>
struct Staged {
  uint4 k[D / 64];
  uint32_t v[2][4];
};

// One block per (128 or 64 rows of a sequence, head, part of their tokens): its
// four waves have a quarter each and share every 64-token step's keys and values, which
// are decoded once on their way into LDS (two buffers: the next step's codes
// are in flight while this one is multiplied).  Decoding per wave instead
// would cost as many vector instructions as the softmax.  Heads run fastest
// over the grid: with 8 heads all blocks of a head share one XCD's L2.
//
// ONE: a step lies in one page (pages of 64 tokens and more), so that its scales
// are two scalars.  Two waves a SIMD cannot hide their own instructions: the
// general form, with four sub-tiles' scales, takes 309 vector and 250 scalar
// instructions a step beside 64 products, and they are its time (two bf16
// prompts of 4096 tokens, 32 query heads of 128, pages of 64: 334 us with it,
// 320 with ONE, 860 TFLOP/s).
template <int DT, int FMT, int D, bool ONE, int RT>
__global__ __launch_bounds__(AT_T, RT == 1 ? (DT == EFFORT_F32 ? 2 : 3) : DT == EFFORT_F32 && D == 128 ? 1 : 2)
void k_attend_prompt(AttendArgs a, float* parts, int32_t tiles, int32_t splits, int32_t out_vec) {
  typedef typename ElemOf<DT>::T T;
  constexpr bool SPLIT = DT == EFFORT_F32;
  constexpr int KS = D / 32, ND = D / 16, SUB = PR_SUB, PR_ROWS = prompt_rows<RT>(), WROWS = 16 * RT;
  __shared__ h8 s_k[2][PR_TILE * D / 8];
  __shared__ h8 s_v[2][PR_TILE * D / 8];
  __shared__ int s_seq;
  const int tid = (int)threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.q_heads / a.kv_heads, shift = __builtin_ctz(a.page_tokens);
  const uint32_t turn = blockIdx.x / (uint32_t)a.kv_heads;
  const int head = (int)(blockIdx.x - turn * (uint32_t)a.kv_heads);
  const int64_t bt = (int64_t)tiles - 1 - turn;  // the last rows see most: they go first
  auto base = [&](int i) { return (int64_t)start_of(a.b, i) * group / PR_ROWS + i; };
  if (tid == 0) s_seq = a.b.seqs;
  __syncthreads();
  for (int i = tid; i < a.b.seqs; i += AT_T)
    if (base(i) <= bt && bt < base(i + 1)) atomicMin(&s_seq, i);
  __syncthreads();
  const int seq = __builtin_amdgcn_readfirstlane(s_seq);
  if (seq >= a.b.seqs) return;
  const int32_t first = start_of(a.b, seq), n = start_of(a.b, seq + 1) - first;
  const int32_t row0 = (int32_t)(bt - base(seq)) * PR_ROWS;
  if (n <= 0 || row0 >= n * group) return;
  const int rows = n * group - row0 < PR_ROWS ? n * group - row0 : PR_ROWS;
  const int64_t len = a.b.lens[seq], cap = (int64_t)a.b.max_pages * a.page_tokens, pos = len - n;
  const int64_t b_min = pos + row0 / group, b_max = pos + (row0 + rows - 1) / group;
  // tokens that the block's rows see
  const int64_t from64 = a.window && b_min + 1 > a.window ? b_min + 1 - a.window : 0;
  int64_t to = b_max + 1 < len ? b_max + 1 : len;
  to = to < cap ? to : cap;
  const int32_t from = from64 < to ? (int32_t)from64 : 0, hi = from64 < to ? (int32_t)to : 0;
  const int32_t lo = from & ~(PR_TILE - 1);
  const int32_t steps = (hi - lo + PR_TILE - 1) / PR_TILE;
  const int32_t z = (int32_t)blockIdx.y;
  const int32_t step0 = (int32_t)((int64_t)steps * z / splits), step1 = (int32_t)((int64_t)steps * (z + 1) / splits);
  const int32_t* table = a.b.table + seq * a.b.table_stride;

  const int last = wave * WROWS + WROWS - 1 < rows ? wave * WROWS + WROWS - 1 : rows - 1;
  const int front = wave * WROWS < rows ? wave * WROWS : rows - 1;
  const int32_t all_high = __builtin_amdgcn_readfirstlane(sight_of(pos + (row0 + front) / group, hi, a.window).high);
  const int32_t all_low = __builtin_amdgcn_readfirstlane(sight_of(pos + (row0 + last) / group, hi, a.window).low);

  f4 o[RT][ND];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[rt][d] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // O counts in `unit`s of the values' scale: a token of scale vs weighs w * vs /
  // unit, with the ratio inside the exponent.  The unit follows the scales up at
  // once, down when they are 2^10 smaller (but never to where what is there
  // could overflow).
  float unit = 0.0f, per_unit = 0.0f, unit_top = 0.0f;
  uint32_t now_vs = 0;  // ONE: the last step's scale, log2 of its ratio to the unit, and 1 / ratio
  float now_up = 0.0f, now_back = 1.0f;
  auto set_unit = [&](float top) {
    unit_top = fmaxf(unit_top, top);
    if (top > 2.0f * unit || (top < 0x1p-10f * unit && top > 0.0f)) {
      const float now = fmaxf(fmaxf(top, unit_top * 0x1p-60f), 0x1p-100f), by = unit / now;
      unit = now;
      per_unit = 1.0f / now;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int d = 0; d < ND; ++d) o[rt][d] *= by;
    }
  };

  // page of the step at t, or of its sub-tile lane & 3; -1: none, behind the
  // block's last step, or a sub-tile before what the rows see, whose page may have
  // any scale
  const int32_t stop = lo + step1 * PR_TILE < hi ? lo + step1 * PR_TILE : hi;
  auto page_at = [&](int32_t t) {
    const int32_t tok = ONE ? t : t + 16 * (lane & 3);
    return tok < stop && (ONE || tok + 15 >= from) ? table[tok >> shift] : -1;
  };
  const int k_piece = tid & (D / 16 - 1), k_tok = tid / (D / 16);  // the first of D / 64 keys, 4096 / D tokens apart
  const int v_el = (tid & (D / 4 - 1)) * 4, v_g = tid / (D / 4) & 3, v_q = wave / (D / 64);
  const bool v_mine = D == 128 || wave < 2;
  const int in_page = (1 << shift) - 1;
  // Addresses are a lane's place in page 0 plus the page times a page's bytes
  // (pages of 16 and 32 tokens divide a step, so that a lane's slot is the same
  // in every step); with ONE a scalar address plus a lane's constant offset.
  // Page 0 is read where there is none, and never used.
  const uint32_t page_bytes = (uint32_t)a.kv_heads << shift << (D == 128 ? 7 : 6);
  const int64_t at_head = (int64_t)head << shift;
  auto lane_base = [&](const uint8_t* c, int tok, int byte) {  // of token `tok` of a step
    return c + (at_head + (tok & in_page)) * D + byte;
  };
  const uint8_t* k_base[D / 64];
  const uint8_t* v_base[2];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) k_base[i] = lane_base(a.kc, k_tok + i * (4096 / D), k_piece * 16);
#pragma unroll
  for (int u = 0; u < 2; ++u) v_base[u] = lane_base(a.vc, (v_q * 2 + u) * 16 + v_g * 4, v_el);
  const float *ks_base = a.ks + head, *vs_base = a.vs + head;
  auto valid = [&](int32_t page) { return (uint32_t)page < (uint32_t)a.b.pages ? (uint32_t)page : 0u; };
  auto fetch = [&](int32_t t, int32_t pages, Staged<D>* st, uint32_t* ks, uint32_t* vs) {
    const uint64_t own = (uint64_t)valid(pages) * (uint32_t)a.kv_heads;
    *ks = __float_as_uint(ks_base[own]);
    *vs = __float_as_uint(vs_base[own]);
    if (ONE) {
      const uint64_t at = (uint64_t)valid(pages) * page_bytes + (uint64_t)(at_head + (t & in_page)) * D;
      const uint8_t *kp = a.kc + at, *vp = a.vc + at;
      const uint32_t k_off = (uint32_t)(k_tok * D + k_piece * 16), v_off = (uint32_t)((v_q * 32 + v_g * 4) * D + v_el);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) st->k[i] = *reinterpret_cast<const uint4*>(kp + (k_off + i * 4096));
      if (v_mine) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) st->v[u][r] = *reinterpret_cast<const uint32_t*>(vp + (v_off + (u * 16 + r) * D));
      }
      return;
    }
    auto place = [&](int sub) {  // of the page of a sub-tile
      return (uint64_t)valid(__builtin_amdgcn_readlane(pages, sub)) * page_bytes;
    };
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int sub = D == 128 ? i * 2 + (wave >> 1) : wave;  // of token k_tok + i * 4096 / D
      st->k[i] = *reinterpret_cast<const uint4*>(k_base[i] + place(sub));
    }
    if (v_mine) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* from_row = v_base[u] + place(v_q * 2 + u);
#pragma unroll
        for (int r = 0; r < 4; ++r) st->v[u][r] = *reinterpret_cast<const uint32_t*>(from_row + r * D);
      }
    }
  };
  auto store = [&](int32_t t, uint32_t ok, Staged<D>& st, uint32_t vs, int buf) {
    // nothing of this may move up to where the codes are still on their way
    asm volatile("" : "+v"(vs));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      asm volatile("" : "+v"(st.k[i].x), "+v"(st.k[i].y), "+v"(st.k[i].z), "+v"(st.k[i].w));
      const int tok = k_tok + i * (4096 / D);
      s_k[buf][key_piece<D>(tok, k_piece * 2)] = decode8<FMT>(st.k[i].x, st.k[i].y);
      s_k[buf][key_piece<D>(tok, k_piece * 2 + 1)] = decode8<FMT>(st.k[i].z, st.k[i].w);
    }
    if (!v_mine) return;
    if (ONE)
      ok = __builtin_amdgcn_readfirstlane(vs) != 0u ? ok : 0u;
    else
      ok &= (uint32_t)__ballot(vs != 0u);
    if ((ok & ((1u << SUB) - 1)) != (1u << SUB) - 1 || t + PR_TILE > hi || t < from) {
      // values of tokens that no row sees weigh 0, so they must not be NaN;
      // those of scale 0 are 0
      int32_t tok0 = t + v_q * 32 + v_g * 4;
      asm volatile("" : "+v"(tok0));
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int32_t tok = tok0 + u * 16 + r;
          if (!(ok >> (v_q * 2 + u) & 1) || tok >= hi || tok < from) st.v[u][r] = 0u;
        }
    }
    uint32_t e[4], e2[4];  // both tokens of a pair: bytes 0 and 1, bytes 2 and 3
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        e[u * 2 + h] = __builtin_amdgcn_perm(st.v[u][2 * h + 1], st.v[u][2 * h], 0x05010400u);
        e2[u * 2 + h] = __builtin_amdgcn_perm(st.v[u][2 * h + 1], st.v[u][2 * h], 0x07030602u);
      }
    const int piece = v_q * 4 + v_g;
    s_v[buf][value_piece<D>(v_el, piece)] =
        join8(decode2<FMT, false>(e[0]), decode2<FMT, false>(e[1]), decode2<FMT, false>(e[2]),
              decode2<FMT, false>(e[3]));
    s_v[buf][value_piece<D>(v_el + 1, piece)] =
        join8(decode2<FMT, true>(e[0]), decode2<FMT, true>(e[1]), decode2<FMT, true>(e[2]), decode2<FMT, true>(e[3]));
    s_v[buf][value_piece<D>(v_el + 2, piece)] = join8(decode2<FMT, false>(e2[0]), decode2<FMT, false>(e2[1]),
                                                      decode2<FMT, false>(e2[2]), decode2<FMT, false>(e2[3]));
    s_v[buf][value_piece<D>(v_el + 3, piece)] =
        join8(decode2<FMT, true>(e2[0]), decode2<FMT, true>(e2[1]), decode2<FMT, true>(e2[2]),
              decode2<FMT, true>(e2[3]));
  };
  auto there = [&](int32_t pages) {  // bit per sub-tile
    const bool in = (uint32_t)pages < (uint32_t)a.b.pages;
    return ONE ? (in ? (1u << SUB) - 1 : 0u) : (uint32_t)__ballot(in) & ((1u << SUB) - 1);
  };

  // Codes of two steps are in flight: those of the next one, which go to LDS
  // during this one, and those of the one after (short prompts have few steps
  // and cold caches: with one step in flight they waited for memory in each).
  // Steps alternate between two sets, in a loop unrolled by two: moving a set
  // would wait for it.
  struct Flight {
    Staged<D> st;
    uint32_t ks, vs, ok;
  };
  Flight even, odd;  // of the steps step0, step0 + 2, ... and the others
  int32_t pages2 = -1;
  // (Behind the last step it reads page 0: with a branch around the loads, the
  // next wait for older ones would wait for these.)
  auto fetch_at = [&](int32_t step, int32_t pages, Flight& to) {
    fetch(lo + step * PR_TILE, pages, &to.st, &to.ks, &to.vs);
    to.ok = there(pages);
  };
  even.ks = even.vs = even.ok = odd.ks = odd.vs = odd.ok = 0;
  if (step0 < step1) {
    const int32_t t = lo + step0 * PR_TILE;
    const int32_t p0 = page_at(t), p1 = page_at(t + PR_TILE), p2 = page_at(t + 2 * PR_TILE);
    fetch_at(step0, p0, even);
    fetch_at(step0 + 1, p1, odd);
    pages2 = p2;
  }
  // this wave's rows (those behind the last one repeat it)
  h8 qh[RT][KS], ql[RT][KS];
  float f[RT];
  Sight see[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    int r = wave * WROWS + rt * 16 + j;
    r = row0 + (r < rows ? r : rows - 1);
    const int i = r / group;
    see[rt] = sight_of(pos + i, hi, a.window);
    const T* src = static_cast<const T*>(a.q) + (first + i) * a.q_stride + (int64_t)(head * group + r - i * group) * D;
    float x[KS][8], top = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) load_n<8>(src + (k * 4 + g) * 8, a.q_vec != 0, x[k]);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[k][e]));
    // the scale's sign goes into q: what is left of it keeps the scores' order
    top = max_of_row(top);
    const float by = power_of_row(top);
    f[rt] = factor_of_row(a.scale, top, by);
    const float mul = a.scale < 0.0f ? -by : by;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= mul;
      qh[rt][k] = weights8(x[k]);
      if (SPLIT) ql[rt][k] = rest8(x[k], qh[rt][k]);
    }
  }
  if (step0 < step1) store(lo + step0 * PR_TILE, even.ok, even.st, even.vs, 0);
  __syncthreads();
  // the lane's pieces of a key by the product, and of a value's tokens by its
  // half; the others lie at constant distances
  int k_at[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) k_at[k] = key_piece<D>(j, k * 4 + g);
  const int v_at[2] = {value_piece<D>(j * ND, g), value_piece<D>(j * ND, 4 + g)};
  // one step: its codes are in LDS buffer `buf` and its scales in `mine`, whose
  // registers then take the step after the next
  auto one_step = [&](int32_t step, int buf, Flight& mine, Flight& next) {
    const int32_t t = lo + step * PR_TILE;
    const uint32_t ks_l = mine.ks, vs_l = mine.vs, ok = mine.ok;
    // the step's scales, those of sub-tile lane & 3 in each lane
    const uint32_t there_now = ok;
    // a poisoned page: its scores are NaN, its values count as any
    const bool bad = ks_l >= 0x7F800000u || vs_l >= 0x7F800000u;
    const float ks_lane = __uint_as_float(bad ? 0x7FC00000u : ks_l);  // (ONE: of the step)
    // 0 where a sub-tile has no say in the unit (values of scale 0 are 0 in LDS)
    const float vs_lane = (ONE ? there_now != 0 : there_now >> (lane & 3) & 1) && !bad ? __uint_as_float(vs_l) : 0.0f;
    float v_hi = vs_lane, v_lo = vs_lane;
    if (!ONE) {
      v_hi = uniform(quad_max(vs_lane));
      v_lo = uniform(-quad_max(vs_lane > 0.0f ? -vs_lane : -INFINITY));
    }
    fetch_at(step + 2, pages2, mine);
    pages2 = page_at(t + 3 * PR_TILE);
    // Sub-tiles whose values' scales are far apart are taken one after the
    // other: the weights of the smaller would lose bits below the larger.
    const int passes = !ONE && v_hi > 0x1p10f * v_lo ? SUB : 1;
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
      const uint32_t here = passes > 1 ? there_now & (1u << pass) : there_now;
      // The fences keep the compiler from loading all pieces at once, for which
      // there are no registers: those of one sub-tile are loaded while the one
      // before is multiplied.
      f4 sc[RT][SUB];
      h8 kf[2][KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) kf[0][k] = s_k[buf][k_at[k]];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        if (u + 1 < SUB) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
            kf[(u + 1) & 1][k] = s_k[buf][k_at[k] + (u + 1) * 16 * (D / 8)];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            sc[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u & 1][k], qh[rt][k], sc[rt][u], 0, 0, 0);
            if (SPLIT) sc[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u & 1][k], ql[rt][k], sc[rt][u], 0, 0, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // scores are sc * c
      float c[RT][SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          c[rt][u] = ONE ? f[rt] * ks_lane : f[rt] * lane_of(ks_lane, u);
      if (here != (1u << SUB) - 1 || t + PR_TILE - 1 > all_high || t <= all_low) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          int32_t high = see[rt].high - t - g * 4, low = see[rt].low - t - g * 4;
          // not to be compared outside this branch: most steps hide nothing
          asm volatile("" : "+v"(high), "+v"(low));
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            sc[rt][u] *= c[rt][u];
            c[rt][u] = 1.0f;
            const int32_t high_u = here >> u & 1 ? high : -PR_TILE;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (16 * u + r > high_u || 16 * u + r <= low) sc[rt][u][r] = -INFINITY;
          }
        }
      }
      float ref[RT], top[RT];
      bool over = false;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        top[rt] = -INFINITY;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          float x = max_of(max_of(max_of(sc[rt][u][0], sc[rt][u][1]), sc[rt][u][2]), sc[rt][u][3]);
          if (!ONE) x *= c[rt][u];
          top[rt] = max_of(top[rt], x);
        }
        top[rt] = max_of_row(ONE ? top[rt] * c[rt][0] : top[rt]);
        over = over || top[rt] > m[rt] + kSlack;
      }
      if (__any(over)) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float mn = fmaxf(top[rt], m[rt]);
          const float alpha = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
          m[rt] = mn;
          l[rt] *= alpha;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[rt][d] *= alpha;
        }
      }
      // nothing seen so far (or only NaN): the weights are 0 (or NaN)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) ref[rt] = kWeightExp - (m[rt] == -INFINITY ? 0.0f : m[rt]);
      if (pass == 0) store(t + PR_TILE, next.ok, next.st, next.vs, buf ^ 1);  // behind the last step: never read
      float up_lane = 0.0f, back_lane = 1.0f;
      if (ONE) {
        if (__float_as_uint(vs_lane) != now_vs) {  // another scale than the last step's
          now_vs = __float_as_uint(vs_lane);
          set_unit(vs_lane);
          const float rel = vs_lane > 0.0f ? vs_lane * per_unit : 1.0f;
          now_up = uniform(__builtin_amdgcn_logf(rel));
          now_back = uniform(__builtin_amdgcn_rcpf(rel));
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) ref[rt] += now_up;
      } else {
        const float vs_here = here >> (lane & 3) & 1 ? vs_lane : 0.0f;
        set_unit(passes > 1 ? uniform(quad_max(vs_here)) : v_hi);
        const float rel = vs_here > 0.0f ? vs_here * per_unit : 1.0f;
        up_lane = __builtin_amdgcn_logf(rel);
        back_lane = __builtin_amdgcn_rcpf(rel);
      }
      float sum[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) sum[rt] = 0.0f;
      h8 ph[RT][2], pl[RT][2];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const float up = ONE ? 0.0f : lane_of(up_lane, u), back = ONE ? 1.0f : lane_of(back_lane, u);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float w[4];
          const float base = ONE ? ref[rt] : ref[rt] + up;
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[rt][u][r], c[rt][u], base));
          if (ONE)
            sum[rt] += (w[0] + w[1]) + (w[2] + w[3]);
          else
            l[rt] = __builtin_fmaf((w[0] + w[1]) + (w[2] + w[3]), back, l[rt]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int e = (u & 1) * 4 + r;
            ph[rt][u >> 1][e] = (_Float16)w[r];
            if (SPLIT) pl[rt][u >> 1][e] = (_Float16)(w[r] - (float)ph[rt][u >> 1][e]);
          }
        }
      }
      if (ONE) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) l[rt] = __builtin_fmaf(sum[rt], now_back, l[rt]);
      }
      __builtin_amdgcn_sched_barrier(0);
      h8 vf[2][4];
      auto load_values = [&](int i, h8* to) {  // products 4 i .. 4 i + 3 of both halves' 2 ND
        const int h = i / (ND / 4), d0 = i % (ND / 4) * 4;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          to[d] = s_v[buf][v_at[h ^ (d0 >> 2)] + (d0 + d) * 16 * (PR_TILE / 8)];
      };
      load_values(0, vf[0]);
#pragma unroll
      for (int i = 0; i < ND / 2; ++i) {
        if (i + 1 < ND / 2) load_values(i + 1, vf[(i + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
        const int h = i / (ND / 4), d0 = i % (ND / 4) * 4;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            f4& acc = o[rt][d0 + d];
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i & 1][d], ph[rt][h], acc, 0, 0, 0);
            if (SPLIT) acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i & 1][d], pl[rt][h], acc, 0, 0, 0);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
  };
#pragma unroll 1
  for (int32_t step = step0; step < step1; step += 2) {
    one_step(step, 0, even, odd);
    if (step + 1 < step1) one_step(step + 1, 1, odd, even);
  }

  // Rows of the result: a lane has the elements (g * 4 + r) * ND + d of row j.
  // They go through LDS, 16 rows of a wave at a time, so that memory sees whole
  // rows: stored from here, 8 bytes of 64 places at a time, they cost as much as
  // a prompt's first hundreds of tokens.
  float* rowbuf = reinterpret_cast<float*>(wave < 2 ? s_k[wave] : s_v[wave - 2]);  // 16 rows of D floats a wave
  static_assert(sizeof(s_k[0]) >= 16 * D * sizeof(float), "a buffer holds a tile of rows");
  float* mine = parts + (((int64_t)bt * a.kv_heads + head) * splits + z) * PR_ROWS * (D + 2);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float sum = sum_of_row(l[rt]);
    const int r0 = wave * WROWS + rt * 16;
    const float by = splits > 1 ? unit : sum == 0.0f ? 0.0f : unit / sum;
    if (splits > 1 && g == 0 && r0 + j < rows) {
      mine[PR_ROWS * D + r0 + j] = m[rt];
      mine[PR_ROWS * D + PR_ROWS + r0 + j] = sum;
    }
    // 16-byte pieces, exchanged by the row so that neighbouring rows fall on different banks
    auto piece = [&](int row, int x) { return row * D + ((x ^ (row & 7)) << 2); };
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int x = 0; x < ND / 4; ++x)
        *reinterpret_cast<f4*>(rowbuf + piece(j, (g * 4 + r) * (ND / 4) + x)) =
            f4{o[rt][x * 4][r], o[rt][x * 4 + 1][r], o[rt][x * 4 + 2][r], o[rt][x * 4 + 3][r]} * by;
    __builtin_amdgcn_wave_barrier();
    constexpr int LANES = D / 4, STEP_ROWS = 64 / LANES;  // lanes of a row
#pragma unroll
    for (int i = 0; i < 16; i += STEP_ROWS) {
      const int r = i + lane / LANES, x = lane % LANES;
      const f4 y = *reinterpret_cast<const f4*>(rowbuf + piece(r, x));
      if (r0 + r >= rows) continue;
      if (splits > 1) {
        *reinterpret_cast<f4*>(mine + (r0 + r) * D + x * 4) = y;
      } else {
        const int row = row0 + r0 + r, tok = row / group;
        T* out = static_cast<T*>(a.out) + (first + tok) * a.out_stride +
                 (int64_t)(head * group + row - tok * group) * D;
        const float v[4] = {y[0], y[1], y[2], y[3]};
        store_n<4>(out + x * 4, out_vec != 0, v);
      }
    }
  }
}

// Joins the parts of k_attend_prompt's rows: one block per (8 rows, head).
template <int DT, int D, int RT>
__global__ __launch_bounds__(AT_T) void k_attend_prompt_join(AttendArgs a, const float* parts, int32_t splits) {
  typedef typename ElemOf<DT>::T T;
  constexpr int PR_ROWS = prompt_rows<RT>();
  __shared__ int s_seq;
  const int tid = (int)threadIdx.x, group = a.q_heads / a.kv_heads, head = (int)blockIdx.x;
  const int64_t bt = blockIdx.y / (PR_ROWS / 8);
  const int r = (int)(blockIdx.y % (PR_ROWS / 8)) * 8 + (tid >> 5);
  auto base = [&](int i) { return (int64_t)start_of(a.b, i) * group / PR_ROWS + i; };
  if (tid == 0) s_seq = a.b.seqs;
  __syncthreads();
  for (int i = tid; i < a.b.seqs; i += AT_T)
    if (base(i) <= bt && bt < base(i + 1)) atomicMin(&s_seq, i);
  __syncthreads();
  const int seq = s_seq;
  if (seq >= a.b.seqs) return;
  const int32_t first = start_of(a.b, seq), n = start_of(a.b, seq + 1) - first;
  const int32_t row = (int32_t)(bt - base(seq)) * PR_ROWS + r;
  if (row >= n * group) return;
  const int tok = row / group;
  T* out = static_cast<T*>(a.out) + (first + tok) * a.out_stride + (int64_t)(head * group + row - tok * group) * D;
  const float* mine = parts + (bt * a.kv_heads + head) * splits * PR_ROWS * (D + 2);
  auto at = [&](int i) { return mine + (int64_t)i * PR_ROWS * (D + 2); };
  join_row<D, 8>(splits, PR_ROWS, r, at, out);
}

// ---------------------------------------------------------------- launches

// Which kernel, by the rows (new tokens times group) of a sequence on average:
// up to 16 or 32 they fit a wave's one or two row tiles and the call is bound
// by reading the cache; beyond that blocks of 64 or 128 rows share what they
// read.  Rows 20 and 32 of 8 sequences of 8000 tokens, bf16: 37 and 39 us with
// two row tiles, 53 and 53 with one at a time, 55 and 60 as prompts; of 32
// sequences: 120 and 124, 211 and 213, 161 and 260.
static int row_tiles(int32_t seqs, int64_t tokens, int32_t group) {
  const int64_t rows = tokens * group;
  return rows <= 16 * (int64_t)seqs ? 1 : rows <= 32 * (int64_t)seqs ? 2 : 0;
}

// Blocks that share a call's chunks.  Two for each CU reach what memory gives; a
// third costs bf16 rows 84.5 us instead of 82.2 (one sequence of 200003 tokens)
// and 212 instead of 199 (64 of 8000), and fp32 rows, which leave no room for
// it, 259 instead of 203.
static int64_t split_blocks() { return 2 * (int64_t)cu_count(); }

// Tables, or windows, of so few tokens: one block of eight waves for each
// item, in some four steps, and nothing to join.  Against the split and its join, fp32
// rows: 8.1 and 11.2 us at 250 tokens of one sequence, 12.2 and 11.1 at 1000;
// 10.4 and 17.2 at 500 of 16, 32.2 and 36.5 at 1000 of 64.  Two row tiles (5
// tokens behind a window of 512, 8 sequences): 14.9 and 22.9, of 64: 42.2 and
// 40.9; of 896, one sequence: 17.8 and 13.9, 64: 55.1 and 48.8, so 640 there.
static int64_t whole_tokens(int rt) { return rt == 2 ? 640 : 1024; }

// How a prompt is shared out: 16-row tiles of a wave, blocks of rows of a head
// (a bound), and in how many parts their tokens are taken so that as many blocks
// as a CU holds fall to every CU.
struct PromptShape {
  int rt;
  int64_t tiles;
  int32_t splits;
};
static PromptShape prompt_of(int rt, int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t group) {
  PromptShape p;
  p.rt = rt;
  p.tiles = tokens * group / (rt == 2 ? prompt_rows<2>() : prompt_rows<1>()) + seqs;
  const int64_t room = (rt == 1 && dim == 64 ? 3 : 2) * (int64_t)cu_count();
  const int64_t z = (room + p.tiles * kv_heads / 2) / (p.tiles * kv_heads);  // the nearest (the tiles are a bound)
  p.splits = (int32_t)(z < 1 ? 1 : z > 32 ? 32 : z);
  return p;
}
// `room`: tokens that a table has room for, all that the host knows of lengths.
// Blocks of 64 rows where there are not two of 128 for each CU (one prompt of 256
// tokens: 13 us, with 128 rows 20; 1024: 30 and 38), but for 1024 rows and more
// before which there may be three times as many tokens: joining more parts of
// larger blocks then costs less (512 tokens behind 4000: 62 us, with 64 rows 81;
// 1024: 110 and 133; 256, of 1024 rows: 43 and 46).  A part has 256 tokens or
// more (64 tokens of one sequence: 9.5 us in one part, 14.9 in as many as fit
// the chip; 256: 13.4 and 15.6).
static PromptShape prompt_shape(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t group,
                                int64_t room) {
  PromptShape p = prompt_of(2, kv_heads, dim, seqs, tokens, group);
  const bool deep = tokens * group >= 1024 * (int64_t)seqs && room * seqs >= 4 * tokens;
  if (p.tiles * kv_heads < 2 * (int64_t)cu_count() && !deep) p = prompt_of(1, kv_heads, dim, seqs, tokens, group);
  const int64_t most = room / 256;
  if (p.splits > most) p.splits = most < 1 ? 1 : (int32_t)most;
  return p;
}

// Enough for any type and any table.
uint64_t attend_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads) {
  if (seqs == 0 || tokens == 0) return 0;
  const int32_t group = q_heads / kv_heads;
  const int rt = row_tiles(seqs, tokens, group);
  if (rt) return (uint64_t)split_blocks() * 2 * (uint64_t)(16 * rt * (dim + 2)) * sizeof(float);
  uint64_t most = 0;
  for (int r = 1; r <= 2; ++r) {
    const PromptShape p = prompt_of(r, kv_heads, dim, seqs, tokens, group);
    const uint64_t rows = (uint64_t)p.tiles * kv_heads * p.splits * (64 * r);
    const uint64_t n = p.splits == 1 ? 0 : rows * (dim + 2) * sizeof(float);
    most = n > most ? n : most;
  }
  return most;
}

template <int DT, int FMT, int D, int RT>
static hipError_t attend_rt(const AttendArgs& a, hipStream_t s) {
  const int64_t nb = split_blocks();
  const int64_t tiles = (int64_t)a.b.tokens * (a.q_heads / a.kv_heads) / (16 * RT) + a.b.seqs;  // of a head, a bound
  float* parts = static_cast<float*>(a.ws);
  int64_t span = (int64_t)a.b.max_pages * a.page_tokens;
  if (a.window && a.window + (int64_t)AT_CHUNK < span) span = a.window + (int64_t)AT_CHUNK;
  if (span <= whole_tokens(RT) && tiles <= 65535) {
    const dim3 grid((unsigned)a.kv_heads, (unsigned)tiles);
    hipLaunchKernelGGL((k_attend_split<DT, FMT, D, RT, 8, true>), grid, dim3(512), 0, s, a, parts);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_attend_split<DT, FMT, D, RT, AT_W, false>), dim3((unsigned)nb), dim3(AT_T), 0, s, a, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // rows of a joining block: one where an item has many parts on average, so
  // that eight groups share them (one sequence of 200000 tokens, 64 parts: 86 us
  // with the split, with four rows 91), four where it has few (16 sequences, 4
  // parts: 6.0 us, with one 11.1)
  const bool many = nb >= 16 * (int64_t)a.b.seqs * a.kv_heads;
  const dim3 grid((unsigned)(tiles * 16 * RT / (many ? 1 : 4)), (unsigned)a.kv_heads);
  if (many)
    hipLaunchKernelGGL((k_attend_join<DT, D, RT, 1>), grid, dim3(AT_T), 0, s, a, parts, (uint32_t)nb);
  else
    hipLaunchKernelGGL((k_attend_join<DT, D, RT, 4>), grid, dim3(AT_T), 0, s, a, parts, (uint32_t)nb);
  return hipGetLastError();
}

template <int DT, int FMT, int D, int RT>
static hipError_t prompt_rt(const AttendArgs& a, const PromptShape& p, hipStream_t s) {
  float* parts = static_cast<float*>(a.ws);
  const int32_t out_vec = rows_aligned<4, typename ElemOf<DT>::T>(a.out, a.out_stride);
  if (p.tiles * a.kv_heads > 0xFFFFFF) return hipErrorInvalidValue;  // 2^32 threads of a dimension
  const int32_t tiles = (int32_t)p.tiles;
  const dim3 grid((unsigned)(p.tiles * a.kv_heads), (unsigned)p.splits);
  if (a.page_tokens >= PR_TILE)
    hipLaunchKernelGGL((k_attend_prompt<DT, FMT, D, true, RT>), grid, dim3(AT_T), 0, s, a, parts, tiles, p.splits,
                       out_vec);
  else
    hipLaunchKernelGGL((k_attend_prompt<DT, FMT, D, false, RT>), grid, dim3(AT_T), 0, s, a, parts, tiles, p.splits,
                       out_vec);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 rows((unsigned)a.kv_heads, (unsigned)(p.tiles * prompt_rows<RT>() / 8));  // splits: few tiles
  hipLaunchKernelGGL((k_attend_prompt_join<DT, D, RT>), rows, dim3(AT_T), 0, s, a, parts, p.splits);
  return hipGetLastError();
}

template <int DT, int FMT, int D>
static hipError_t attend_prompt(const AttendArgs& a, hipStream_t s) {
  const PromptShape p = prompt_shape(a.kv_heads, D, a.b.seqs, a.b.tokens, a.q_heads / a.kv_heads,
                                     (int64_t)a.b.max_pages * a.page_tokens);
  return p.rt == 1 ? prompt_rt<DT, FMT, D, 1>(a, p, s) : prompt_rt<DT, FMT, D, 2>(a, p, s);
}

template <int DT, int FMT, int D>
static hipError_t attend_rows(const AttendArgs& a, hipStream_t s) {
  switch (row_tiles(a.b.seqs, a.b.tokens, a.q_heads / a.kv_heads)) {
    case 1: return attend_rt<DT, FMT, D, 1>(a, s);
    case 2: return attend_rt<DT, FMT, D, 2>(a, s);
    default: return attend_prompt<DT, FMT, D>(a, s);
  }
}

template <int DT, int FMT>
static hipError_t attend_dim(const AttendArgs& a, hipStream_t s) {
  return a.dim == 64 ? attend_rows<DT, FMT, 64>(a, s) : attend_rows<DT, FMT, 128>(a, s);
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
