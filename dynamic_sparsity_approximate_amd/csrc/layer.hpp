// layer.hpp -- argument blocks and launchers of the kernels between a decoder
// layer's matvecs (kv_append.hpp, kv_attend.hpp, norm.hip), and of what several
// continuations of a sequence need (kv_pages.hip, beam.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "effort.h"

namespace effort {

// Where the new tokens of a call belong (effort_kv_batch), as the kernels read it.
struct BatchArgs {
  const int32_t* table;   // [seqs][max_pages], rows table_stride apart
  const int32_t* lens;    // [seqs]
  const int32_t* starts;  // [seqs + 1]
  int64_t table_stride;
  int64_t pages;
  int32_t seqs, max_pages, tokens;
};

struct AppendArgs {
  BatchArgs b;
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, q_out_stride, k_stride, v_stride;
  const float* rope;  // [rows][rot / 2][2]
  uint8_t *kc, *vc;
  float *ks, *vs;
  int32_t rot, interleaved, q_heads, kv_heads, dim, page_tokens, format;
  // launch_append_ex: each may be null
  const int32_t* parents;
  const void *q_norm, *k_norm;  // [dim], of head h at h * stride
  int64_t q_norm_stride, k_norm_stride;
  double eps;
};

struct AttendArgs {
  BatchArgs b;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  float scale;
  int32_t window, q_heads, kv_heads, dim, page_tokens, format;
  int32_t q_vec;  // q's rows are aligned to 8 elements
  void* ws;
  const int32_t* parents;  // launch_attend_tree
};

// The caches of a model's layers, as many as a launch takes.
#define EFFORT_KV_SET 64
struct CacheArgs {
  uint8_t *k, *v;
  float *ks, *vs;
  int32_t heads, dim, format, unused;
};
struct CacheSet {
  CacheArgs c[EFFORT_KV_SET];
  int64_t pages;
  int32_t count, page_tokens;
};

// effort_kv_book
struct BookArgs {
  int32_t *table, *lens, *refs, *info;
  int64_t table_stride, pages;
  int32_t seqs, max_pages, page_tokens;
};

struct BeamArgs {
  const void* logits;
  int64_t stride;  // elements between rows
  const float* scores;
  const uint8_t* ended;
  int32_t items, beams, vocab, keep, end_token;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  void* ws;
};

struct NormArgs {
  const void *x, *resid, *post_w, *gate, *pre_w;
  void *resid_out, *out;
  int64_t rows, n, x_stride, resid_stride, gate_stride, resid_out_stride, out_stride;
  float scale, eps;
};

hipError_t launch_rope_table(double base, int64_t rows, int32_t rot, float* table, hipStream_t s);
hipError_t launch_append(const AppendArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_append_ex(const AppendArgs& a, int32_t dtype, hipStream_t s);
uint64_t attend_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads);
hipError_t launch_attend(const AttendArgs& a, int32_t dtype, hipStream_t s);
uint64_t tree_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads);
hipError_t launch_attend_tree(const AttendArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_fork(const BookArgs& b, const int32_t* source, const int32_t* keep, hipStream_t s);
uint64_t grow_workspace(const BookArgs& b);
hipError_t launch_grow(const BookArgs& b, const effort_kv_cache* caches, int32_t count, const int32_t* more_of,
                       int32_t more, void* ws, hipStream_t s);
hipError_t launch_copy(const effort_kv_cache* caches, int32_t count, int64_t n, const int32_t* from, const int32_t* to,
                       hipStream_t s);
uint64_t accept_workspace(int32_t seqs);
hipError_t launch_accept(const effort_kv_cache* caches, int32_t count, const BatchArgs& b, const int32_t* parents,
                         const int32_t* leaf, int32_t* lens_out, void* ws, hipStream_t s);
uint64_t beam_workspace(int64_t rows, int64_t vocab);
hipError_t launch_beam(const BeamArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, int32_t dtype, int32_t resid_dtype, hipStream_t s);

}  // namespace effort
