// Host-side declarations of the cross-attention and cache operators.
#pragma once

#include "ress_internal.h"

namespace ress {

constexpr int kMaxSeqs = 8192;   // sequences, requests

// Validated shape of ress_cross_attn and ress_cross_attn_bwd.
struct CrossGeometry {
  int nq, nk, seqs, heads, kv_heads, group;
  long long q_stride, k_stride, v_stride;   // elements between token rows
};

// Arguments of the attention kernels: keys either packed (k, v) or paged codes.
struct CrossParams {
  DeviceError* err;
  int nq, nk, seqs, heads, kv_heads, group;
  long long q_stride, k_stride, v_stride;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* q_off;    // NULL: one sequence of all rows
  const int32_t* k_off;
  const int32_t* q_lens;   // NULL: no padding
  const int32_t* k_lens;
  __nv_bfloat16* out;
  float* lse;              // [heads][nq] or NULL
  // The cache.
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lengths;
  int pages, page, max_pages, step;
};

struct CrossBwdParams {
  DeviceError* err;
  int nq, nk, seqs, heads, kv_heads, group;
  long long q_stride, k_stride, v_stride;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* out;
  const __nv_bfloat16* dout;
  const float* lse;
  const int32_t* q_off;
  const int32_t* k_off;
  const int32_t* q_lens;
  const int32_t* k_lens;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
};

size_t cross_workspace(const CrossGeometry& g);
size_t cross_bwd_workspace(const CrossGeometry& g);
size_t cache_attn_workspace(const ress_cache_shape& s, int heads, int tokens);
ress_status launch_cross(CrossParams p, void* ws, cudaStream_t st);
ress_status launch_cross_bwd(const CrossGeometry& g, CrossBwdParams p, void* ws, cudaStream_t st);
ress_status launch_cache_attn(CrossParams p, void* ws, cudaStream_t st);
size_t cache_decode_workspace();
ress_status launch_cache_decode(const CrossParams& c, void* ws, cudaStream_t st);

ress_status launch_cache_plan(const ress_cache_shape& s, const int32_t* added,
                              const int32_t* lengths, int32_t* table, const int32_t* free_pages,
                              int32_t n_free, const int32_t* cursor, int32_t tokens,
                              int32_t* offsets, int32_t* slots, int32_t* new_lengths,
                              int32_t* new_cursor, cudaStream_t st);
ress_status launch_cache_append(const ress_cache_shape& s, const void* k, const void* v, bool f32,
                                int64_t k_stride, int64_t v_stride, const int32_t* slots,
                                int32_t tokens, void* k_cache, void* v_cache, float* k_scale,
                                float* v_scale, cudaStream_t st);

}  // namespace ress
