// layer.hpp -- argument blocks and launchers of the kernels between a decoder
// layer's matvecs (kv_append.hip, kv_attend.hip, norm.hip).
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
};

struct NormArgs {
  const void *x, *resid, *post_w, *gate, *pre_w;
  void *resid_out, *out;
  int64_t rows, n, x_stride, resid_stride, gate_stride, resid_out_stride, out_stride;
  float scale, eps;
};

hipError_t launch_rope_table(double base, int64_t rows, int32_t rot, float* table, hipStream_t s);
hipError_t launch_append(const AppendArgs& a, int32_t dtype, hipStream_t s);
uint64_t attend_workspace(int32_t kv_heads, int32_t dim, int32_t seqs, int64_t tokens, int32_t q_heads);
hipError_t launch_attend(const AttendArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, int32_t dtype, int32_t resid_dtype, hipStream_t s);

}  // namespace effort
