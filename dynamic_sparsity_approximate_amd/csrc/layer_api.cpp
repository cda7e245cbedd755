// layer_api.cpp -- C ABI of what lies between a decoder layer's matvecs, and of several
// continuations of a sequence: argument validation and launches.  Every check happens before the first enqueue.
#include <hip/hip_runtime.h>
#include <math.h>

#include "effort.h"
#include "host.hpp"
#include "layer.hpp"

using namespace effort;

namespace {

constexpr int64_t kMaxTokens = 1ll << 24;
constexpr int64_t kMaxNorm = 1ll << 20;
constexpr int64_t kMaxVocab = 1ll << 20;  // tokens count in 20 bits
constexpr int64_t kMaxIndex = 0x7FFFFFFFll;
constexpr int64_t kMaxLength = 1ll << 30;  // kernels step past a length in 32 bits
constexpr int32_t kMaxKvHeads = 256, kMaxGroup = 64;

uintptr_t bytes_of(int32_t dtype) { return dtype == EFFORT_F32 ? 4 : 2; }
bool dtype_ok(int32_t d) { return d == EFFORT_F32 || d == EFFORT_F16 || d == EFFORT_BF16; }

// Sizes of a cache that the host alone can judge (no pointers).
bool cache_sizes_ok(const effort_kv_cache* c) {
  return c && (c->format == EFFORT_KV_E4M3 || c->format == EFFORT_KV_I8) && c->kv_heads >= 1 &&
         c->kv_heads <= kMaxKvHeads && (c->head_dim == 64 || c->head_dim == 128) &&
         (c->page_tokens == 16 || c->page_tokens == 32 || c->page_tokens == 64 || c->page_tokens == 128);
}

bool cache_ok(const effort_kv_cache* c) {
  return cache_sizes_ok(c) && c->pages >= 1 && c->pages <= kMaxIndex && c->k && c->v && c->k_scale &&
         c->v_scale && aligned(c->k, 16) && aligned(c->v, 16) && aligned(c->k_scale, 4) &&
         aligned(c->v_scale, 4);
}

// A call with no sequences or no tokens has nothing to do: its arrays may be null.
bool batch_ok(const effort_kv_batch* b, int32_t page_tokens) {
  if (!b || b->seqs < 0 || b->seqs > EFFORT_KV_MAX_SEQS || b->tokens < 0 || b->tokens > kMaxTokens)
    return false;
  if (b->seqs == 0 || b->tokens == 0) return true;
  return b->max_pages >= 1 && (int64_t)b->max_pages * page_tokens <= kMaxLength &&
         b->table_stride >= b->max_pages && b->page_table && b->kv_lens && b->q_starts &&
         aligned(b->page_table, 4) && aligned(b->kv_lens, 4) && aligned(b->q_starts, 4);
}

BatchArgs batch_args(const effort_kv_batch* b, int64_t pages) {
  BatchArgs a;
  a.table = b->page_table;
  a.lens = b->kv_lens;
  a.starts = b->q_starts;
  a.table_stride = b->table_stride;
  a.pages = pages;
  a.seqs = b->seqs;
  a.max_pages = b->max_pages;
  a.tokens = (int32_t)b->tokens;
  return a;
}

bool rows_ok(const void* p, int64_t stride, int64_t width, uintptr_t bytes) {
  return p && aligned(p, bytes) && stride >= width;
}

bool page_tokens_ok(int32_t t) { return t == 16 || t == 32 || t == 64 || t == 128; }

bool book_ok(const effort_kv_book* b) {
  if (!b || b->seqs < 0 || b->seqs > EFFORT_KV_MAX_SEQS || b->reserved != 0 || !page_tokens_ok(b->page_tokens))
    return false;
  if (b->max_pages < 1 || (int64_t)b->max_pages * b->page_tokens > kMaxLength || b->table_stride < b->max_pages ||
      b->pages < 1 || b->pages > kMaxIndex)
    return false;
  if (b->seqs == 0) return true;
  return b->page_table && b->kv_lens && b->refs && b->info && aligned(b->page_table, 4) && aligned(b->kv_lens, 4) &&
         aligned(b->refs, 4) && aligned(b->info, 4);
}

BookArgs book_args(const effort_kv_book* b) {
  return BookArgs{b->page_table, b->kv_lens, b->refs, b->info, b->table_stride, b->pages, b->seqs, b->max_pages,
                  b->page_tokens};
}

// Caches of one number of pages and one page_tokens.
bool caches_ok(const effort_kv_cache* c, int32_t count) {
  if (count < 0 || count > EFFORT_KV_MAX_CACHES || (count > 0 && !c)) return false;
  for (int32_t i = 0; i < count; ++i)
    if (!cache_ok(c + i) || c[i].pages != c[0].pages || c[i].page_tokens != c[0].page_tokens) return false;
  return true;
}

// 0, or why the workspace does not do.
int space_of(const void* ws, uint64_t bytes, uint64_t need) {
  if (need && (!ws || !aligned(ws, 256))) return EFFORT_EINVAL;
  return bytes < need ? EFFORT_ENOSPACE : EFFORT_OK;
}

bool beam_sizes_ok(int64_t items, int32_t beams, int64_t vocab) {
  return items >= 0 && items <= kMaxTokens && beams >= 1 && beams <= EFFORT_BEAM_MAX && items * beams <= kMaxTokens &&
         vocab >= 1 && vocab <= kMaxVocab;
}

bool heads_ok(int32_t q_heads, int32_t kv_heads) {
  return q_heads >= 1 && q_heads % kv_heads == 0 && q_heads / kv_heads <= kMaxGroup;
}

}  // namespace

extern "C" {

int effort_rope_table(double base, int64_t rows, int32_t rot_dim, float* table_dev, void* stream) {
  if (!table_dev || !aligned(table_dev, 8) || rows < 1 || rows > kMaxIndex) return EFFORT_EINVAL;
  if (rot_dim < 8 || rot_dim > 128 || rot_dim % 8 || !(base > 1.0) || !isfinite(base)) return EFFORT_EINVAL;
  return status_of(launch_rope_table(base, rows, rot_dim, table_dev, static_cast<hipStream_t>(stream)));
}

int effort_kv_append_ex(const effort_kv_cache* cache, const effort_kv_batch* batch, const int32_t* parents_dev,
                        int32_t dtype, const float* rope_dev, int64_t rope_rows, int32_t rot_dim,
                        int32_t interleaved, const void* q_norm_dev, int64_t q_norm_stride,
                        const void* k_norm_dev, int64_t k_norm_stride, double eps, const void* q_dev,
                        int64_t q_stride, int32_t q_heads, void* q_out_dev, int64_t q_out_stride,
                        const void* k_dev, int64_t k_stride, const void* v_dev, int64_t v_stride, void* stream) {
  if (!cache_ok(cache) || !batch_ok(batch, cache->page_tokens) || !dtype_ok(dtype)) return EFFORT_EINVAL;
  if (interleaved != 0 && interleaved != 1) return EFFORT_EINVAL;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 8) return EFFORT_EINVAL;
  if (q_dev && !heads_ok(q_heads, cache->kv_heads)) return EFFORT_EINVAL;
  if (!(eps >= 0.0) || !isfinite(eps) || !aligned(parents_dev, 4)) return EFFORT_EINVAL;
  for (int64_t stride : {q_norm_dev ? q_norm_stride : 0, k_norm_dev ? k_norm_stride : 0})
    if (stride != 0 && stride < cache->head_dim) return EFFORT_EINVAL;
  if (!aligned(q_norm_dev, bytes_of(dtype)) || !aligned(k_norm_dev, bytes_of(dtype))) return EFFORT_EINVAL;
  if (batch->seqs == 0 || batch->tokens == 0) return EFFORT_OK;
  if (rot_dim && (!rope_dev || !aligned(rope_dev, 8) ||
                  rope_rows < (int64_t)batch->max_pages * cache->page_tokens))
    return EFFORT_EINVAL;
  const uintptr_t es = bytes_of(dtype);
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (!rows_ok(k_dev, k_stride, row, es) || !rows_ok(v_dev, v_stride, row, es)) return EFFORT_EINVAL;
  if (q_dev) {
    const int64_t qrow = (int64_t)q_heads * cache->head_dim;
    if (!rows_ok(q_dev, q_stride, qrow, es) || !rows_ok(q_out_dev, q_out_stride, qrow, es))
      return EFFORT_EINVAL;
    if (q_out_dev == q_dev && q_out_stride != q_stride) return EFFORT_EINVAL;
  }
  AppendArgs a;
  a.b = batch_args(batch, cache->pages);
  a.q = q_dev;
  a.k = k_dev;
  a.v = v_dev;
  a.q_out = q_out_dev;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.rope = rope_dev;
  a.kc = cache->k;
  a.vc = cache->v;
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.q_heads = q_dev ? q_heads : 0;
  a.kv_heads = cache->kv_heads;
  a.dim = cache->head_dim;
  a.page_tokens = cache->page_tokens;
  a.format = cache->format;
  a.parents = parents_dev;
  a.q_norm = q_dev ? q_norm_dev : nullptr;
  a.k_norm = k_norm_dev;
  a.q_norm_stride = q_norm_stride;
  a.k_norm_stride = k_norm_stride;
  a.eps = eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool plain = !parents_dev && !a.q_norm && !a.k_norm;
  return status_of(plain ? launch_append(a, dtype, s) : launch_append_ex(a, dtype, s));
}

int effort_kv_append(const effort_kv_cache* cache, const effort_kv_batch* batch, int32_t dtype,
                     const float* rope_dev, int64_t rope_rows, int32_t rot_dim, int32_t interleaved,
                     const void* q_dev, int64_t q_stride, int32_t q_heads, void* q_out_dev,
                     int64_t q_out_stride, const void* k_dev, int64_t k_stride, const void* v_dev,
                     int64_t v_stride, void* stream) {
  return effort_kv_append_ex(cache, batch, nullptr, dtype, rope_dev, rope_rows, rot_dim, interleaved, nullptr, 0,
                             nullptr, 0, 0.0, q_dev, q_stride, q_heads, q_out_dev, q_out_stride, k_dev, k_stride,
                             v_dev, v_stride, stream);
}

int effort_kv_workspace_bytes(const effort_kv_cache* cache, int32_t seqs, int64_t tokens,
                              int32_t q_heads, uint64_t* bytes) {
  if (!bytes || !cache_sizes_ok(cache) || seqs < 0 || seqs > EFFORT_KV_MAX_SEQS || tokens < 0 ||
      tokens > kMaxTokens || !heads_ok(q_heads, cache->kv_heads))
    return EFFORT_EINVAL;
  *bytes = attend_workspace(cache->kv_heads, cache->head_dim, seqs, tokens, q_heads);
  return EFFORT_OK;
}

// parents_dev NULL: no trees.
static int attention(const effort_kv_cache* cache, const effort_kv_batch* batch, const int32_t* parents_dev,
                     int32_t dtype, const void* q_dev, int64_t q_stride, int32_t q_heads, float scale,
                     int32_t window, void* out_dev, int64_t out_stride, void* ws_dev, uint64_t ws_bytes,
                     void* stream) {
  if (!cache_ok(cache) || !batch_ok(batch, cache->page_tokens) || !dtype_ok(dtype)) return EFFORT_EINVAL;
  if (!heads_ok(q_heads, cache->kv_heads) || !isfinite(scale) || window < 0) return EFFORT_EINVAL;
  if (batch->seqs == 0 || batch->tokens == 0) return EFFORT_OK;
  const uintptr_t es = bytes_of(dtype);
  const int64_t row = (int64_t)q_heads * cache->head_dim;
  if (!rows_ok(q_dev, q_stride, row, es) || !rows_ok(out_dev, out_stride, row, es)) return EFFORT_EINVAL;
  if (out_dev == q_dev) return EFFORT_EINVAL;
  const uint64_t need = (parents_dev ? tree_workspace : attend_workspace)(
      cache->kv_heads, cache->head_dim, batch->seqs, batch->tokens, q_heads);
  if (need && (!ws_dev || !aligned(ws_dev, 256))) return EFFORT_EINVAL;
  if (ws_bytes < need) return EFFORT_ENOSPACE;
  AttendArgs a;
  a.b = batch_args(batch, cache->pages);
  a.q = q_dev;
  a.out = out_dev;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.kc = cache->k;
  a.vc = cache->v;
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.scale = scale;
  a.window = window;
  a.q_heads = q_heads;
  a.kv_heads = cache->kv_heads;
  a.dim = cache->head_dim;
  a.page_tokens = cache->page_tokens;
  a.format = cache->format;
  a.q_vec = aligned(q_dev, 8 * es) && q_stride % 8 == 0;
  a.ws = ws_dev;
  a.parents = parents_dev;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return status_of(parents_dev ? launch_attend_tree(a, dtype, s) : launch_attend(a, dtype, s));
}

int effort_kv_tree_workspace_bytes(const effort_kv_cache* cache, int32_t seqs, int64_t tokens,
                                   int32_t q_heads, uint64_t* bytes) {
  if (!bytes || !cache_sizes_ok(cache) || seqs < 0 || seqs > EFFORT_KV_MAX_SEQS || tokens < 0 ||
      tokens > kMaxTokens || !heads_ok(q_heads, cache->kv_heads))
    return EFFORT_EINVAL;
  *bytes = tree_workspace(cache->kv_heads, cache->head_dim, seqs, tokens, q_heads);
  return EFFORT_OK;
}

int effort_kv_attention(const effort_kv_cache* cache, const effort_kv_batch* batch, int32_t dtype,
                        const void* q_dev, int64_t q_stride, int32_t q_heads, float scale,
                        int32_t window, void* out_dev, int64_t out_stride, void* ws_dev,
                        uint64_t ws_bytes, void* stream) {
  return attention(cache, batch, nullptr, dtype, q_dev, q_stride, q_heads, scale, window, out_dev, out_stride, ws_dev,
                   ws_bytes, stream);
}

int effort_kv_attention_tree(const effort_kv_cache* cache, const effort_kv_batch* batch,
                             const int32_t* parents_dev, int32_t dtype, const void* q_dev, int64_t q_stride,
                             int32_t q_heads, float scale, int32_t window, void* out_dev, int64_t out_stride,
                             void* ws_dev, uint64_t ws_bytes, void* stream) {
  // with nothing to do the arrays may be null
  if ((!parents_dev && batch && batch->seqs > 0 && batch->tokens > 0) || !aligned(parents_dev, 4)) return EFFORT_EINVAL;
  return attention(cache, batch, parents_dev, dtype, q_dev, q_stride, q_heads, scale, window, out_dev, out_stride,
                   ws_dev, ws_bytes, stream);
}

int effort_kv_fork(const effort_kv_book* book, const int32_t* source_dev, const int32_t* lens_dev, void* stream) {
  if (!book_ok(book)) return EFFORT_EINVAL;
  if (book->seqs == 0) return EFFORT_OK;
  if (!source_dev || !aligned(source_dev, 4) || !aligned(lens_dev, 4)) return EFFORT_EINVAL;
  return status_of(launch_fork(book_args(book), source_dev, lens_dev, static_cast<hipStream_t>(stream)));
}

int effort_kv_grow_workspace_bytes(const effort_kv_book* book, uint64_t* bytes) {
  if (!bytes || !book_ok(book)) return EFFORT_EINVAL;
  *bytes = grow_workspace(book_args(book));
  return EFFORT_OK;
}

int effort_kv_grow(const effort_kv_book* book, const effort_kv_cache* caches, int32_t count,
                   const int32_t* more_dev, int32_t more, void* ws_dev, uint64_t ws_bytes, void* stream) {
  if (!book_ok(book) || !caches_ok(caches, count) || !aligned(more_dev, 4)) return EFFORT_EINVAL;
  if (count > 0 && (caches[0].pages != book->pages || caches[0].page_tokens != book->page_tokens))
    return EFFORT_EINVAL;
  if (book->seqs == 0) return EFFORT_OK;
  const BookArgs b = book_args(book);
  const int bad = space_of(ws_dev, ws_bytes, grow_workspace(b));
  if (bad) return bad;
  return status_of(launch_grow(b, caches, count, more_dev, more, ws_dev, static_cast<hipStream_t>(stream)));
}

int effort_kv_copy_pages(const effort_kv_cache* caches, int32_t count, const int32_t* from_dev,
                         const int32_t* to_dev, int64_t n, void* stream) {
  if (!caches_ok(caches, count) || n < 0 || n > kMaxIndex) return EFFORT_EINVAL;
  if (count == 0 || n == 0) return EFFORT_OK;
  if (!from_dev || !to_dev || !aligned(from_dev, 4) || !aligned(to_dev, 4)) return EFFORT_EINVAL;
  return status_of(launch_copy(caches, count, n, from_dev, to_dev, static_cast<hipStream_t>(stream)));
}

int effort_kv_accept_workspace_bytes(int32_t seqs, uint64_t* bytes) {
  if (!bytes || seqs < 0 || seqs > EFFORT_KV_MAX_SEQS) return EFFORT_EINVAL;
  *bytes = accept_workspace(seqs);
  return EFFORT_OK;
}

int effort_kv_accept(const effort_kv_cache* caches, int32_t count, const effort_kv_batch* batch,
                     const int32_t* parents_dev, const int32_t* leaf_dev, int32_t* lens_out_dev, void* ws_dev,
                     uint64_t ws_bytes, void* stream) {
  if (count < 1 || !caches_ok(caches, count) || !batch_ok(batch, caches[0].page_tokens)) return EFFORT_EINVAL;
  if (batch->seqs == 0) return EFFORT_OK;
  if (batch->tokens == 0 && (!batch->kv_lens || !batch->q_starts || !batch->page_table)) return EFFORT_EINVAL;
  if (!leaf_dev || !lens_out_dev || !aligned(leaf_dev, 4) || !aligned(lens_out_dev, 4) || !aligned(parents_dev, 4))
    return EFFORT_EINVAL;
  if (parents_dev) {
    const int bad = space_of(ws_dev, ws_bytes, accept_workspace(batch->seqs));
    if (bad) return bad;
  }
  return status_of(launch_accept(caches, count, batch_args(batch, caches[0].pages), parents_dev, leaf_dev, lens_out_dev,
                                 ws_dev, static_cast<hipStream_t>(stream)));
}

int effort_beam_workspace_bytes(int64_t items, int32_t beams, int64_t vocab, uint64_t* bytes) {
  if (!bytes || !beam_sizes_ok(items, beams, vocab)) return EFFORT_EINVAL;
  *bytes = items == 0 ? 0 : beam_workspace(items * beams, vocab);
  return EFFORT_OK;
}

int effort_beam_select(int32_t dtype, const void* logits_dev, int64_t stride, const float* scores_dev,
                       const uint8_t* ended_dev, int32_t end_token, int64_t items, int32_t beams, int64_t vocab,
                       int32_t keep, float* out_scores_dev, int32_t* out_parents_dev, int32_t* out_tokens_dev,
                       void* ws_dev, uint64_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || !beam_sizes_ok(items, beams, vocab) || keep < 1 || keep > EFFORT_BEAM_MAX_KEEP)
    return EFFORT_EINVAL;
  if (items == 0) return EFFORT_OK;  // nothing to do: the arrays may be null
  if (!rows_ok(logits_dev, stride, vocab, bytes_of(dtype)) || !scores_dev || !aligned(scores_dev, 4))
    return EFFORT_EINVAL;
  for (const void* p : {(const void*)out_scores_dev, (const void*)out_parents_dev, (const void*)out_tokens_dev})
    if (!p || !aligned(p, 4)) return EFFORT_EINVAL;
  const int bad = space_of(ws_dev, ws_bytes, beam_workspace(items * beams, vocab));
  if (bad) return bad;
  BeamArgs a;
  a.logits = logits_dev;
  a.stride = stride;
  a.scores = scores_dev;
  a.ended = ended_dev;
  a.items = (int32_t)items;
  a.beams = beams;
  a.vocab = (int32_t)vocab;
  a.keep = keep;
  a.end_token = end_token;
  a.out_scores = out_scores_dev;
  a.out_parents = out_parents_dev;
  a.out_tokens = out_tokens_dev;
  a.ws = ws_dev;
  return status_of(launch_beam(a, dtype, static_cast<hipStream_t>(stream)));
}

int effort_norm_residual(int32_t dtype, int64_t rows, int64_t n, const void* x_dev, int64_t x_stride,
                         int32_t resid_dtype, const void* resid_dev, int64_t resid_stride,
                         const void* post_w_dev, const void* gate_dev, int64_t gate_stride,
                         float scale, const void* pre_w_dev, float eps, void* resid_out_dev,
                         int64_t resid_out_stride, void* out_dev, int64_t out_stride, void* stream) {
  if (!dtype_ok(dtype) || (resid_dtype != dtype && resid_dtype != EFFORT_F32)) return EFFORT_EINVAL;
  if (rows < 0 || rows > kMaxIndex || n < 1 || n > kMaxNorm || !(eps >= 0.0f) || !isfinite(eps))
    return EFFORT_EINVAL;
  if (rows == 0) return EFFORT_OK;  // nothing to do: the arrays may be null
  if (!resid_out_dev && !out_dev) return EFFORT_EINVAL;
  const uintptr_t es = bytes_of(dtype), rs = bytes_of(resid_dtype);
  if (!rows_ok(x_dev, x_stride, n, es)) return EFFORT_EINVAL;
  if (resid_dev && !rows_ok(resid_dev, resid_stride, n, rs)) return EFFORT_EINVAL;
  if (resid_out_dev && !rows_ok(resid_out_dev, resid_out_stride, n, rs)) return EFFORT_EINVAL;
  if (out_dev && !rows_ok(out_dev, out_stride, n, es)) return EFFORT_EINVAL;
  if (gate_dev && (!aligned(gate_dev, es) || (gate_stride != 0 && gate_stride < n))) return EFFORT_EINVAL;
  if (!aligned(post_w_dev, es) || !aligned(pre_w_dev, es)) return EFFORT_EINVAL;
  if (resid_out_dev && resid_out_dev == resid_dev && resid_out_stride != resid_stride) return EFFORT_EINVAL;
  if (out_dev && out_dev == x_dev && out_stride != x_stride) return EFFORT_EINVAL;
  if (out_dev && (out_dev == resid_dev || out_dev == resid_out_dev)) return EFFORT_EINVAL;
  if (resid_out_dev && resid_out_dev == x_dev) return EFFORT_EINVAL;
  NormArgs a;
  a.x = x_dev;
  a.resid = resid_dev;
  a.post_w = post_w_dev;
  a.gate = gate_dev;
  a.pre_w = pre_w_dev;
  a.resid_out = resid_out_dev;
  a.out = out_dev;
  a.rows = rows;
  a.n = n;
  a.x_stride = x_stride;
  a.resid_stride = resid_stride;
  a.gate_stride = gate_stride;
  a.resid_out_stride = resid_out_stride;
  a.out_stride = out_stride;
  a.scale = scale;
  a.eps = eps;
  return status_of(launch_norm(a, dtype, resid_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
