// kv_pages.hip -- who holds the pages of a cache: sequences that continue others (fork), room
// for new tokens (grow), copies of pages, and the accepted path of a tree (accept).
//
// Everything here is a matter of latency and of copied bytes.  Tables and counts are small:
// a fork is one launch (2.2 us for 4 sequences, 4 for 16 after 81 MB of copies), a growth
// one block (5.2 us) and the copies that it asks for.  Every result is
// the same whatever the order of blocks: counts change by commuting atomics only, and pages
// are given out in order, the lowest first.
#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "host.hpp"
#include "layer.hpp"
#include "tree.hpp"

namespace effort {

constexpr int PG_T = 1024, PG_W = PG_T / 64;
static_assert(EFFORT_KV_MAX_SEQS <= PG_T, "a thread for each sequence");

__device__ inline bool is_page(int32_t p, int64_t pages) { return p >= 0 && p < pages; }

// ---------------------------------------------------------------- fork

// Entries of a block's columns of all sequences, in LDS.
constexpr int FK_ENTRIES = 16384, FK_COLS = 64, FK_BLOCKS = 1 << 16;

// New entry (s, c) is the old (source[s], c) where that is in front of the new end, so that
// columns are independent: a block reads its columns of every sequence before it writes any.
// The lengths are everybody's: the last block that has read them writes them.
__global__ __launch_bounds__(PG_T) void k_fork(BookArgs b, const int32_t* source, const int32_t* keep, int cols_log) {
  __shared__ int32_t s_old[FK_ENTRIES];
  __shared__ int32_t s_src[EFFORT_KV_MAX_SEQS], s_len[EFFORT_KV_MAX_SEQS];
  __shared__ int s_last;
  const int tid = (int)threadIdx.x, cols = 1 << cols_log, n = b.seqs << cols_log;
  if (tid < b.seqs) {
    const int32_t src = source[tid];
    const bool ok = src >= 0 && src < b.seqs;
    int32_t len = ok ? b.lens[src] : 0;
    if (keep && keep[tid] < len) len = keep[tid];
    s_src[tid] = ok ? src : -1;
    s_len[tid] = len < 0 ? 0 : len;
  }
  for (int32_t col0 = (int32_t)blockIdx.x << cols_log; col0 < b.max_pages; col0 += (int32_t)gridDim.x << cols_log) {
    for (int i = tid; i < n; i += PG_T) {
      const int32_t c = col0 + (i & (cols - 1));
      s_old[i] = c < b.max_pages ? b.table[(i >> cols_log) * b.table_stride + c] : -1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += PG_T) {
      const int s = i >> cols_log, c = i & (cols - 1);
      if (col0 + c >= b.max_pages) continue;
      int32_t now = -1;
      if (s_src[s] >= 0 && (int64_t)(col0 + c) * b.page_tokens < s_len[s]) now = s_old[(s_src[s] << cols_log) + c];
      if (!is_page(now, b.pages)) now = -1;
      const int32_t old = s_old[i];
      if (now == old) continue;
      b.table[s * b.table_stride + col0 + c] = now;
      if (is_page(old, b.pages)) atomicSub(b.refs + old, 1);
      if (now >= 0) atomicAdd(b.refs + now, 1);
    }
    __syncthreads();
  }
  if (tid == 0) {
    s_last = 1;
    if (gridDim.x > 1) {
      // (every thread's lengths are in LDS since the barrier)
      const int32_t t = __hip_atomic_fetch_add(b.info + 1, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      s_last = t == (int32_t)gridDim.x - 1;
      if (s_last) __hip_atomic_store(b.info + 1, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __syncthreads();
  if (s_last && tid < b.seqs) b.lens[tid] = s_len[tid];
}

hipError_t launch_fork(const BookArgs& b, const int32_t* source, const int32_t* keep, hipStream_t s) {
  int cols_log = 0;
  while ((1 << cols_log) < FK_COLS && (b.seqs << (cols_log + 1)) <= FK_ENTRIES) ++cols_log;
  const int64_t blocks = ((int64_t)b.max_pages + (1 << cols_log) - 1) >> cols_log;
  // tables of more columns than blocks: a launch has less than 2^32 threads
  const unsigned grid = (unsigned)(blocks < FK_BLOCKS ? blocks : FK_BLOCKS);
  hipLaunchKernelGGL(k_fork, dim3(grid), dim3(PG_T), 0, s, b, source, keep, cols_log);
  return hipGetLastError();
}

// ---------------------------------------------------------------- grow

// What k_grow leaves for k_copy: pages to copy, and how many of their first slots.
struct Copy {
  int32_t from, to, slots, unused;
};
// Workspace: `count` and the copies, then the free pages that are given out and what they replace.
struct GrowSpace {
  int32_t* count;
  Copy* copies;
  int32_t *free, *old;
};
static int64_t most_new(const BookArgs& b) {
  const int64_t n = (int64_t)b.seqs * b.max_pages;
  return n < b.pages ? n : b.pages;
}
static GrowSpace space_of(const BookArgs& b, void* ws) {
  GrowSpace g;
  g.count = static_cast<int32_t*>(ws);
  g.copies = reinterpret_cast<Copy*>(g.count + 4);
  g.free = reinterpret_cast<int32_t*>(g.copies + b.seqs);
  g.old = g.free + most_new(b);
  return g;
}
uint64_t grow_workspace(const BookArgs& b) { return 16 + (uint64_t)b.seqs * sizeof(Copy) + 8 * (uint64_t)most_new(b); }

// Sum over the threads in front of this one; *total: over all.  s_w: PG_W words, free again on return.
__device__ inline int64_t scan(int64_t x, int64_t* s_w, int64_t* total) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  int64_t run = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) s_w[wave] = run;
  __syncthreads();
  int64_t before = run - x, all = 0;
  for (int w = 0; w < PG_W; ++w) {
    if (w < wave) before += s_w[w];
    all += s_w[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

// One block: what is given out depends on what was before.  Bound by its chain of reads:
// lengths, table, counts; the first 16384 pages' counts come with them, and where every
// sequence needs one column at most, as in decoding, and these pages have room, all is settled
// between three barriers (16 sequences: 5.2 us, by the general way 10.7).  The general way
// reads all counts from page 0 until it has found enough: a fork and a growth of 16
// sequences take 16 us, a call of each, while the first pages are free, 42 where the first
// 40000 are held, 67 with 90000 and 98 with 160000.
// A sequence's new tokens need the columns from len / page_tokens on.  The first
// may hold older tokens; if others hold that page, too, it is copied, but by the last of this
// call's sequences if the call has all its holders.  Another column keeps a page that it has
// alone.  What is needed is counted, then the lowest free pages are found, and only if there
// are enough of them does anything change.
__global__ __launch_bounds__(PG_T) void k_grow(BookArgs b, const int32_t* more_of, int32_t more, GrowSpace ws) {
  __shared__ int64_t s_w[PG_W];
  __shared__ int64_t s_start[EFFORT_KV_MAX_SEQS + 1];  // columns before a sequence's
  __shared__ int32_t s_first[EFFORT_KV_MAX_SEQS];      // its first column
  // the page of it that holds older tokens; -1: none does, -2: an absent one
  __shared__ int32_t s_page[EFFORT_KV_MAX_SEQS];
  __shared__ uint8_t s_copy[EFFORT_KV_MAX_SEQS];
  __shared__ int32_t s_count;
  __shared__ int32_t s_free[EFFORT_KV_MAX_SEQS];
  const int tid = (int)threadIdx.x, T = b.page_tokens, lane = tid & 63, wave = tid >> 6;
  const bool mine = tid < b.seqs;
  // the first pages' counts, on their way with all that leads to what is needed
  constexpr int U = 16;
  uint32_t free0 = 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tid * U + u < b.pages && b.refs[tid * U + u] == 0) free0 |= 1u << u;
  int64_t len = 0, add = 0, beyond = 0, columns = 0;
  int32_t page = -1, first = 0;
  int part = 0;
  if (tid == 0) s_count = 0;
  if (mine) {
    len = b.lens[tid];
    add = more_of ? more_of[tid] : more;
    len = len < 0 ? 0 : len;
    add = add < 0 ? 0 : add;
    const int64_t c0 = len / T, c1 = (len + add + T - 1) / T;  // columns [c0, c1)
    if (add > 0) {
      const int64_t end = c1 < b.max_pages ? c1 : b.max_pages;
      columns = c0 < end ? end - c0 : 0;
      beyond = c1 - c0 - columns;
      first = (int32_t)(c0 < b.max_pages ? c0 : b.max_pages);
      part = (int)(len - c0 * T);
      if (part > 0 && columns > 0) {
        page = b.table[tid * b.table_stride + first];
        if (!is_page(page, b.pages)) page = -2;
      }
    }
    s_first[tid] = first;
    s_page[tid] = page;
  }
  auto copies_page = [&]() {  // whether this thread's sequence copies its page (s_page is complete)
    const int32_t held = page >= 0 ? b.refs[page] : 0;
    if (held <= 1) return false;
    int here = 0;
    bool later = false;
    for (int s = 0; s < b.seqs; ++s)
      if (s_page[s] == page) {
        ++here;
        later = later || s > tid;
      }
    return later || here < held;
  };
  // A column each, and pages enough among the first 16384: what decoding asks for.  (A
  // prompt's growth, or one that these pages do not suffice for, begins anew below.)
  if (!__syncthreads_or(columns > 1 || beyond > 0)) {
    int32_t entry = -1;
    bool need = false, copy = false;
    if (columns > 0) {
      copy = copies_page();
      if (page == -1) {
        entry = b.table[tid * b.table_stride + first];
        need = !(is_page(entry, b.pages) && b.refs[entry] <= 1);
      } else {
        entry = page;
        need = copy;
      }
    }
    const uint64_t needs = __ballot(need);
    int run = __popc(free0);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(run, d);
      if (lane >= d) run += o;
    }
    if (lane == 63) s_w[wave] = (int64_t)run << 32 | (uint32_t)__popcll(needs);
    __syncthreads();
    int rank = __popcll(needs & ((1ull << lane) - 1)), at = run - __popc(free0);
    int want = 0, found = 0;
#pragma unroll
    for (int w = 0; w < PG_W; ++w) {
      const int nw = (int)(uint32_t)s_w[w], fw = (int)(s_w[w] >> 32);
      if (w < wave) rank += nw;
      if (w < wave) at += fw;
      want += nw;
      found += fw;
    }
    if (found >= want) {
      for (uint32_t f = free0; f && at < want; f &= f - 1) s_free[at++] = tid * U + __builtin_ctz(f);
      __syncthreads();
      if (need) {
        const int32_t now = s_free[rank];
        b.table[tid * b.table_stride + first] = now;
        b.refs[now] = 1;
        if (is_page(entry, b.pages)) atomicSub(b.refs + entry, 1);
        if (copy) ws.copies[atomicAdd(&s_count, 1)] = Copy{entry, now, part, 0};
      }
      if (mine) b.lens[tid] = (int32_t)(len + add < 0x7FFFFFFF ? len + add : 0x7FFFFFFF);
      __syncthreads();
      if (tid == 0) {
        b.info[0] = 0;
        *ws.count = s_count;
      }
      return;
    }
    __syncthreads();
  }
  int64_t total, missing;
  const int64_t start = scan(columns, s_w, &total);  // (its barriers publish s_page, too)
  scan(beyond, s_w, &missing);
  if (mine) {
    s_start[tid] = start;
    s_copy[tid] = copies_page();
  }
  if (tid == 0) s_start[b.seqs] = total;
  __syncthreads();

  // item i: a column of a sequence; whether it needs a page
  auto place = [&](int64_t i, int* s, int32_t* col, int32_t* entry) {
    int lo = 0, hi = b.seqs;  // the last sequence that starts at or before i: it has columns
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= i) lo = mid; else hi = mid;
    }
    *s = lo;
    *col = s_first[lo] + (int32_t)(i - s_start[lo]);
    *entry = b.table[lo * b.table_stride + *col];
    // (an absent page whose older tokens are lost stays absent)
    if (*col == s_first[lo] && s_page[lo] != -1) return s_copy[lo] != 0;
    return !(is_page(*entry, b.pages) && b.refs[*entry] <= 1);
  };
  int64_t needed = 0;
  for (int64_t i0 = 0; i0 < total; i0 += PG_T) {
    int s;
    int32_t col, entry;
    needed += i0 + tid < total && place(i0 + tid, &s, &col, &entry);
  }
  int64_t want;
  scan(needed, s_w, &want);

  // the lowest free pages, 16 of a thread at a time
  int64_t found = 0;
  for (int64_t p0 = 0; p0 < b.pages && found < want; p0 += (int64_t)PG_T * U) {
    const int64_t p = p0 + (int64_t)tid * U;
    uint32_t free = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p + u < b.pages && b.refs[p + u] == 0) free |= 1u << u;
    int64_t here;
    int64_t at = found + scan(__popc(free), s_w, &here);
    for (; free && at < want; free &= free - 1) ws.free[at++] = (int32_t)(p + __builtin_ctz(free));
    found += here;
  }
  missing += want > found ? want - found : 0;
  if (missing > 0) {  // nothing changes
    if (tid == 0) {
      b.info[0] = missing < 0x7FFFFFFF ? (int32_t)missing : 0x7FFFFFFF;
      *ws.count = 0;
    }
    return;
  }
  __syncthreads();  // the list of free pages is this block's own, in memory
  int64_t rank = 0;
  for (int64_t i0 = 0; i0 < total && want > 0; i0 += PG_T) {
    int s = 0;
    int32_t col = 0, entry = -1;
    const bool need = i0 + tid < total && place(i0 + tid, &s, &col, &entry);
    int64_t here;
    const int64_t at = rank + scan(need, s_w, &here);
    if (need) {
      const int32_t now = ws.free[at];
      b.table[s * b.table_stride + col] = now;
      ws.old[at] = is_page(entry, b.pages) ? entry : -1;
      if (col == s_first[s] && s_page[s] >= 0)
        ws.copies[atomicAdd(&s_count, 1)] = Copy{entry, now, (int32_t)(b.lens[s] % T), 0};
    }
    rank += here;
  }
  __syncthreads();  // counts change when all have been read
  for (int64_t i = tid; i < want; i += PG_T) {
    b.refs[ws.free[i]] = 1;
    if (ws.old[i] >= 0) atomicSub(b.refs + ws.old[i], 1);
  }
  if (mine) b.lens[tid] = (int32_t)(len + add < 0x7FFFFFFF ? len + add : 0x7FFFFFFF);
  if (tid == 0) {
    b.info[0] = 0;
    *ws.count = s_count;
  }
}

// ---------------------------------------------------------------- copies

constexpr int CY_T = 256;

// A wave copies one head's codes of a page, keys or values, and its scale, 8 KB at a time.
// Nothing of it is used again before the caches have seen much else, so that it passes them
// by (10 copies of 62 tokens in 32 layers' caches of 8 heads of 128, 81 MB read and written:
// 19.6 us, 4.1 TB/s; with ordinary loads and stores 26.7).  blockIdx.y: the cache.
typedef uint32_t Piece __attribute__((ext_vector_type(4)));
// `most`: pairs that there is room for; what pair(i) is for a later i than the last does
// not matter.  The first pair comes with their number.
template <typename Count, typename Pair>
__device__ inline void copy_planes(const CacheSet& set, int64_t most, Count count, Pair pair) {
  const CacheArgs& c = set.c[blockIdx.y];
  const int lane = (int)threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * (CY_T / 64);
  const uint32_t planes = 2 * (uint32_t)c.heads;
  const int64_t plane = (int64_t)set.page_tokens * c.dim;
  uint32_t wave = blockIdx.x * (CY_T / 64) + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t at = wave / planes;
  Copy p = pair(at < most ? at : most - 1);
  const int64_t all = count() * planes;
  for (int64_t i = wave; i < all; i += waves) {
    if (i != wave) {
      at = i / planes;
      p = pair(at);
    }
    const int ph = (int)(i - at * planes), head = ph >> 1;
    if (!is_page(p.from, set.pages) || !is_page(p.to, set.pages) || p.from == p.to) continue;
    uint8_t* codes = (ph & 1) ? c.v : c.k;
    float* scale = (ph & 1) ? c.vs : c.ks;
    const Piece* from = reinterpret_cast<const Piece*>(codes + ((int64_t)p.from * c.heads + head) * plane);
    Piece* to = reinterpret_cast<Piece*>(codes + ((int64_t)p.to * c.heads + head) * plane);
    const int pieces = p.slots * c.dim / 16;  // 1024 at most
    constexpr int U = 8;
    for (int j0 = 0; j0 < pieces; j0 += 64 * U) {
      Piece x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u * 64 + lane < pieces) x[u] = __builtin_nontemporal_load(from + j0 + u * 64 + lane);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u * 64 + lane < pieces) __builtin_nontemporal_store(x[u], to + j0 + u * 64 + lane);
    }
    if (lane == 0) scale[(int64_t)p.to * c.heads + head] = scale[(int64_t)p.from * c.heads + head];
  }
}

__global__ __launch_bounds__(CY_T) void k_copy_grown(CacheSet set, int32_t most, const int32_t* count,
                                                      const Copy* copies) {
  copy_planes(set, most, [&]() { return (int64_t)*count; }, [&](int64_t i) { return copies[i]; });
}

__global__ __launch_bounds__(CY_T) void k_copy(CacheSet set, int64_t count, const int32_t* from, const int32_t* to) {
  copy_planes(set, count, [&]() { return count; }, [&](int64_t i) { return Copy{from[i], to[i], set.page_tokens, 0}; });
}

// Blocks of a cache for at most `most` pages: a wave for each plane, up to what fills the chip.
static unsigned copy_blocks(const CacheSet& set, int64_t most) {
  int heads = 1;
  for (int i = 0; i < set.count; ++i) heads = set.c[i].heads > heads ? set.c[i].heads : heads;
  const int64_t blocks = (most * 2 * heads + CY_T / 64 - 1) / (CY_T / 64);
  const int64_t full = (8 * (int64_t)cu_count() + set.count - 1) / set.count;
  return (unsigned)(blocks < full ? blocks : full);
}

// `run` for at most EFFORT_KV_SET caches at a time.
template <typename Run>
static hipError_t each_set(const effort_kv_cache* caches, int32_t count, Run run) {
  for (int32_t i = 0; i < count; i += EFFORT_KV_SET) {
    CacheSet set;
    set.count = count - i < EFFORT_KV_SET ? count - i : EFFORT_KV_SET;
    set.page_tokens = caches[0].page_tokens;
    set.pages = caches[0].pages;
    for (int32_t j = 0; j < set.count; ++j) {
      const effort_kv_cache& c = caches[i + j];
      set.c[j] = CacheArgs{c.k, c.v, c.k_scale, c.v_scale, c.kv_heads, c.head_dim, c.format, 0};
    }
    run(set);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_grow(const BookArgs& b, const effort_kv_cache* caches, int32_t count, const int32_t* more_of,
                       int32_t more, void* ws, hipStream_t s) {
  const GrowSpace g = space_of(b, ws);
  hipLaunchKernelGGL(k_grow, dim3(1), dim3(PG_T), 0, s, b, more_of, more, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return each_set(caches, count, [&](const CacheSet& set) {
    hipLaunchKernelGGL(k_copy_grown, dim3(copy_blocks(set, b.seqs), (unsigned)set.count), dim3(CY_T), 0, s, set,
                       b.seqs, g.count, g.copies);
  });
}

hipError_t launch_copy(const effort_kv_cache* caches, int32_t count, int64_t n, const int32_t* from, const int32_t* to,
                       hipStream_t s) {
  return each_set(caches, count, [&](const CacheSet& set) {
    hipLaunchKernelGGL(k_copy, dim3(copy_blocks(set, n), (unsigned)set.count), dim3(CY_T), 0, s, set, n, from, to);
  });
}

// ---------------------------------------------------------------- accept

// A sequence's accepted path: `count` tokens from position `base` on, the first `still` of
// them in place; token i is the sequence's new token path[i].
struct Path {
  int32_t base, count, still, unused;
  int16_t path[EFFORT_KV_MAX_TREE];
};
uint64_t accept_workspace(int32_t seqs) { return (uint64_t)seqs * sizeof(Path); }

// One wave per sequence: walks from the leaf up, and writes the new length.
__global__ __launch_bounds__(64) void k_path(BatchArgs b, int32_t page_tokens, const int32_t* parents,
                                             const int32_t* leaf, int32_t* lens_out, Path* paths) {
  __shared__ int16_t s_up[EFFORT_KV_MAX_TREE], s_path[EFFORT_KV_MAX_TREE];
  const int s = (int)blockIdx.x, lane = (int)threadIdx.x;
  const int32_t first = start_of(b, s), len = b.lens[s], T = page_tokens;
  const int64_t n = (int64_t)start_of(b, s + 1) - first, base = (int64_t)len - n;
  const int32_t* table = b.table + s * b.table_stride;
  Path* out = paths + s;
  int32_t last = leaf[s];
  if (last >= n) last = -1;
  if (n <= 0 || base < 0 || (parents && !is_tree(n, base))) {
    if (lane == 0) {
      lens_out[s] = len;
      if (paths) out->count = out->still = 0;
    }
    return;
  }
  int32_t count = last < 0 ? 0 : last + 1;
  if (parents && last >= 0) {
    for (int i = lane; i <= last; i += 64) s_up[i] = up_of(parents[first + i], i);
    __syncthreads();
    count = depth_of(s_up, last) + 1;
    if (lane == 0) {
      int i = count - 1;
      for (int p = last; p >= 0; p = s_up[p]) s_path[i--] = (int16_t)p;
    }
    __syncthreads();
  }
  // a path ends in front of the first token that is in no page
  auto in_page = [&](int64_t pos) { return pos / T < b.max_pages && is_page(table[pos / T], b.pages); };
  int32_t cut = count, still = count;
  if (parents) {
    for (int i = lane; i < count; i += 64) {
      const int a = s_path[i];
      if (!in_page(base + a) || !in_page(base + i)) cut = i < cut ? i : cut;
      if (a != i) still = i < still ? i : still;
    }
  } else {
    for (int64_t c = base / T + lane; c * T < base + count; c += 64)
      if (!in_page(c * T)) {
        const int32_t at = c * T > base ? (int32_t)(c * T - base) : 0;
        cut = at < cut ? at : cut;
      }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const int32_t c = __shfl_xor(cut, d), t = __shfl_xor(still, d);
    cut = c < cut ? c : cut;
    still = t < still ? t : still;
  }
  if (paths) {
    for (int i = lane; i < cut; i += 64) out->path[i] = s_path[i];
    if (lane == 0) {
      out->base = (int32_t)base;
      out->count = cut;
      out->still = still < cut ? still : cut;
    }
  }
  if (lane == 0) lens_out[s] = (int32_t)(base + cut);
}

// Codes of the values code * from: nearest codes to them in units of `now`.
template <int FMT>
__device__ inline uint32_t requant(uint32_t w, double from, double now) {
  float y[4];
  const double most = FMT == EFFORT_KV_I8 ? 127.0 : 448.0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const double x = (double)decode<FMT>(w >> (8 * j) & 0xFFu) * from / now;
    y[j] = now > 0.0 ? round_to_odd(__builtin_fmin(__builtin_fmax(x, -most), most)) : 0.0f;
  }
  return encode4<FMT>(y[0], y[1], y[2], y[3]);
}

// The least power of two, at least 2^EFFORT_KV_MIN_EXP, whose largest code takes x > 0.
template <int FMT>
__device__ inline float scale_for(double x) {
  const double most = FMT == EFFORT_KV_I8 ? 127.0 : 448.0;
  int e;
  (void)frexp(x / most, &e);  // x / most in [2^(e - 1), 2^e), but for its rounding
  e -= 2;
  while (x > ldexp(most, e)) ++e;  // exact: most has 7 bits
  return ldexpf(1.0f, e < EFFORT_KV_MIN_EXP ? EFFORT_KV_MIN_EXP : e > 127 ? 127 : e);
}

// One wave's part: a head's keys or values of a sequence.  Bound by the chain path, table,
// codes: paths of eight trees in 32 layers' caches of 8 heads, 1.6 MB read and written, take
// 8.2 us and the walk in front of them 4.  Pages of the path are taken in
// order, and a page's tokens in order, as many at a time as 16-byte pieces fit a wave: a
// token comes from a slot at or behind its own, so that nothing is overwritten before it
// is read.  A page's scale grows where a token from another page needs it; then all of the
// page's tokens become the nearest codes, as in an append.
template <int FMT>
__device__ void move_path(const CacheArgs& c, int32_t T, uint8_t* codes, float* scales, int head, const Path& path,
                          const int32_t* table) {
  const int lane = (int)threadIdx.x & 63, row = c.dim / 16, per = 64 / row, piece = lane % row;
  auto scale_at = [&](int32_t page) { return scales + (int64_t)page * c.heads + head; };
  auto codes_at = [&](int32_t page, int slot) {
    return reinterpret_cast<uint4*>(codes + (((int64_t)page * c.heads + head) * T + slot) * c.dim) + piece;
  };
  auto bad = [](float x) { return __float_as_uint(x) >= 0x7F800000u; };  // negative ones, too
  int i0 = 0;
  while (i0 < path.count) {
    const int32_t to_page = table[(path.base + i0) / T];
    const int slot0 = (path.base + i0) % T;
    const int i1 = path.count < i0 + T - slot0 ? path.count : i0 + T - slot0;
    const float old = *scale_at(to_page);
    double top = 0.0;
    bool poison = false;
    for (int i = i0; i < i1; i += per) {
      const int k = i + lane / row;
      if (k >= i1) continue;
      const int32_t at = path.base + path.path[k], page = table[at / T];
      if (page == to_page) continue;
      const float s = *scale_at(page);
      const uint4 x = *codes_at(page, at % T);
      poison = poison || bad(s);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) most = fmaxf(most, fabsf(decode<FMT>(w[j >> 2] >> (8 * (j & 3)) & 0xFFu)));
      top = __builtin_fmax(top, (double)most * (double)s);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = __builtin_fmax(top, __shfl_xor(top, d));
    poison = __any(poison);
    float now = old;
    if (poison && !bad(old)) now = __uint_as_float(0x7FC00000u);
    if (!poison && !bad(old) && top > 0.0) {
      const float need = scale_for<FMT>(top);
      now = need > old ? need : old;
    }
    const bool raised = !poison && now > old;
    if (lane == 0 && (raised || (poison && !bad(old)))) *scale_at(to_page) = now;
    if (raised)
      for (int i = 0; i < slot0; i += per) {
        const int slot = i + lane / row;
        if (slot >= slot0) continue;
        uint4* p = codes_at(to_page, slot);
        uint4 x = *p;
        x.x = requant<FMT>(x.x, old, now);
        x.y = requant<FMT>(x.y, old, now);
        x.z = requant<FMT>(x.z, old, now);
        x.w = requant<FMT>(x.w, old, now);
        *p = x;
      }
    for (int i = i0; i < i1; i += per) {
      const int k = i + lane / row;
      if (k >= i1) continue;
      const int a = path.path[k];
      const int32_t at = path.base + a, page = table[at / T];
      if (a == k && !raised) continue;
      uint4 x = *codes_at(page, at % T);
      if (page != to_page || raised) {
        const double s = page == to_page ? (double)old : (double)*scale_at(page);
        if (poison || bad(now)) {
          if (page != to_page) x = uint4{0u, 0u, 0u, 0u};
        } else {
          x.x = requant<FMT>(x.x, s, now);
          x.y = requant<FMT>(x.y, s, now);
          x.z = requant<FMT>(x.z, s, now);
          x.w = requant<FMT>(x.w, s, now);
        }
      }
      *codes_at(to_page, (path.base + k) % T) = x;
    }
    i0 = i1;
  }
}

__global__ __launch_bounds__(CY_T) void k_move(CacheSet set, BatchArgs b, const Path* paths) {
  const CacheArgs& c = set.c[blockIdx.y];
  const int s = (int)blockIdx.z;
  const int ph = (int)blockIdx.x * (CY_T / 64) + ((int)threadIdx.x >> 6), head = ph >> 1;
  const Path& path = paths[s];
  if (path.still == path.count || head >= c.heads) return;
  const int32_t* table = b.table + s * b.table_stride;
  uint8_t* codes = (ph & 1) ? c.v : c.k;
  float* scales = (ph & 1) ? c.vs : c.ks;
  if (c.format == EFFORT_KV_I8)
    move_path<EFFORT_KV_I8>(c, set.page_tokens, codes, scales, head, path, table);
  else
    move_path<EFFORT_KV_E4M3>(c, set.page_tokens, codes, scales, head, path, table);
}

hipError_t launch_accept(const effort_kv_cache* caches, int32_t count, const BatchArgs& b, const int32_t* parents,
                         const int32_t* leaf, int32_t* lens_out, void* ws, hipStream_t s) {
  Path* paths = parents ? static_cast<Path*>(ws) : nullptr;
  hipLaunchKernelGGL(k_path, dim3((unsigned)b.seqs), dim3(64), 0, s, b, caches[0].page_tokens, parents, leaf, lens_out,
                     paths);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !paths) return e;
  return each_set(caches, count, [&](const CacheSet& set) {
    int heads = 1;
    for (int i = 0; i < set.count; ++i) heads = set.c[i].heads > heads ? set.c[i].heads : heads;
    const dim3 grid((unsigned)((2 * heads + CY_T / 64 - 1) / (CY_T / 64)), (unsigned)set.count, (unsigned)b.seqs);
    hipLaunchKernelGGL(k_move, grid, dim3(CY_T), 0, s, set, b, paths);
  });
}

}  // namespace effort
