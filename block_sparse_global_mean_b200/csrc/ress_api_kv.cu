// C ABI of the cross-attention and cache operators: host-side argument checks
// and workspace queries.  Every entry point validates before its first CUDA
// call.
#include "ress_common.cuh"
#include "ress_kv.h"

namespace ress {
namespace {

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

constexpr int64_t kMaxTokens = (int64_t)1 << 30;

// Row stride in elements (0: dense rows of `width`); 0 back when it is invalid.
long long row_stride(int64_t stride, int64_t width, int unit) {
  if (stride == 0) return width;
  return stride >= width && stride % unit == 0 && stride <= ((int64_t)1 << 32) ? stride : 0;
}

ress_status check_heads(int32_t heads, int32_t kv_heads, int32_t head_dim) {
  if (heads <= 0 || kv_heads <= 0 || head_dim <= 0 || heads % kv_heads != 0)
    return RESS_ERR_INVALID_ARG;
  return head_dim == kHeadDim && heads <= kMaxHeads ? RESS_OK : RESS_ERR_UNSUPPORTED;
}

ress_status check_cross(const ress_cross_shape* s, CrossGeometry* g) {
  if (s == nullptr || s->nq < 0 || s->nk < 0 || s->seqs <= 0) return RESS_ERR_INVALID_ARG;
  if (ress_status e = check_heads(s->heads, s->kv_heads, s->head_dim)) return e;
  if (s->dtype != RESS_BF16)
    return s->dtype == RESS_F32 ? RESS_ERR_UNSUPPORTED : RESS_ERR_INVALID_ARG;
  if (s->nq > kMaxTokens || s->nk > kMaxTokens || s->seqs > kMaxSeqs) return RESS_ERR_UNSUPPORTED;
  g->nq = (int)s->nq;
  g->nk = (int)s->nk;
  g->seqs = s->seqs;
  g->heads = s->heads;
  g->kv_heads = s->kv_heads;
  g->group = s->heads / s->kv_heads;
  g->q_stride = row_stride(s->q_stride, (int64_t)s->heads * kHeadDim, 8);
  g->k_stride = row_stride(s->k_stride, (int64_t)s->kv_heads * kHeadDim, 8);
  g->v_stride = row_stride(s->v_stride, (int64_t)s->kv_heads * kHeadDim, 8);
  return g->q_stride && g->k_stride && g->v_stride ? RESS_OK : RESS_ERR_INVALID_ARG;
}

// Offsets: both or neither; without them there is one sequence.  Lengths are
// optional by themselves.
ress_status check_seq_arrays(const CrossGeometry& g, const int32_t* q_offsets,
                             const int32_t* kv_offsets, const int32_t* q_lens,
                             const int32_t* kv_lens) {
  if ((q_offsets == nullptr) != (kv_offsets == nullptr)) return RESS_ERR_INVALID_ARG;
  if (q_offsets == nullptr && g.seqs != 1) return RESS_ERR_INVALID_ARG;
  if (!aligned(q_offsets, 4) || !aligned(kv_offsets, 4) || !aligned(q_lens, 4) ||
      !aligned(kv_lens, 4))
    return RESS_ERR_INVALID_ARG;
  return RESS_OK;
}

ress_status check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (need == 0) return RESS_OK;
  if (workspace == nullptr || bytes < need) return RESS_ERR_WORKSPACE;
  return aligned(workspace, 256) ? RESS_OK : RESS_ERR_INVALID_ARG;
}

ress_status check_pool(const ress_cache_shape* s, bool heads) {
  if (s == nullptr || s->pages <= 0 || s->page <= 0) return RESS_ERR_INVALID_ARG;
  if (heads) {
    if (ress_status e = check_heads(s->kv_heads, s->kv_heads, s->head_dim)) return e;
  }
  if (s->page != 64 && s->page != 128) return RESS_ERR_UNSUPPORTED;
  return (int64_t)s->pages * s->page < ((int64_t)1 << 31) ? RESS_OK : RESS_ERR_UNSUPPORTED;
}

ress_status check_table(const ress_cache_shape* s) {
  if (s->requests <= 0 || s->max_pages <= 0) return RESS_ERR_INVALID_ARG;
  if (s->requests > kMaxSeqs || (int64_t)s->max_pages * s->page >= ((int64_t)1 << 31))
    return RESS_ERR_UNSUPPORTED;
  return RESS_OK;
}

}  // namespace
}  // namespace ress

using namespace ress;

extern "C" {

size_t ress_cross_workspace_bytes(const ress_cross_shape* shape) {
  CrossGeometry g;
  return check_cross(shape, &g) == RESS_OK ? cross_workspace(g) : 0;
}

size_t ress_cross_bwd_workspace_bytes(const ress_cross_shape* shape) {
  CrossGeometry g;
  return check_cross(shape, &g) == RESS_OK ? cross_bwd_workspace(g) : 0;
}

ress_status ress_cross_attn(const ress_cross_shape* shape, const void* q, const void* k,
                            const void* v, const int32_t* q_offsets, const int32_t* kv_offsets,
                            const int32_t* q_lens, const int32_t* kv_lens, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  CrossGeometry g;
  if (ress_status s = check_cross(shape, &g)) return s;
  if (ress_status s = check_seq_arrays(g, q_offsets, kv_offsets, q_lens, kv_lens)) return s;
  if (g.nq == 0) return RESS_OK;
  if (!q || !out || (g.nk > 0 && (!k || !v))) return RESS_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return RESS_ERR_INVALID_ARG;
  if (ress_status s = check_workspace(cross_workspace(g), workspace, workspace_bytes)) return s;
  CrossParams p{};
  if ((p.err = device_error_ptr()) == nullptr) return RESS_ERR_CUDA;
  p.nq = g.nq;
  p.nk = g.nk;
  p.seqs = g.seqs;
  p.heads = g.heads;
  p.kv_heads = g.kv_heads;
  p.group = g.group;
  p.q_stride = g.q_stride;
  p.k_stride = g.k_stride;
  p.v_stride = g.v_stride;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_off = q_offsets;
  p.k_off = kv_offsets;
  p.q_lens = q_lens;
  p.k_lens = kv_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  return launch_cross(p, workspace, static_cast<cudaStream_t>(stream));
}

ress_status ress_cross_attn_bwd(const ress_cross_shape* shape, const void* q, const void* k,
                                const void* v, const void* out, const float* lse,
                                const void* dout, const int32_t* q_offsets,
                                const int32_t* kv_offsets, const int32_t* q_lens,
                                const int32_t* kv_lens, void* dq, void* dk, void* dv,
                                void* workspace, size_t workspace_bytes, void* stream) {
  CrossGeometry g;
  if (ress_status s = check_cross(shape, &g)) return s;
  if (ress_status s = check_seq_arrays(g, q_offsets, kv_offsets, q_lens, kv_lens)) return s;
  if (g.nq == 0 && g.nk == 0) return RESS_OK;
  if (g.nq > 0 && (!q || !out || !lse || !dout || !dq)) return RESS_ERR_INVALID_ARG;
  if (g.nk > 0 && (!k || !v || !dk || !dv)) return RESS_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(lse, 4))
    return RESS_ERR_INVALID_ARG;
  if (ress_status s = check_workspace(cross_bwd_workspace(g), workspace, workspace_bytes))
    return s;
  CrossBwdParams p{};
  if ((p.err = device_error_ptr()) == nullptr) return RESS_ERR_CUDA;
  p.nq = g.nq;
  p.nk = g.nk;
  p.seqs = g.seqs;
  p.heads = g.heads;
  p.kv_heads = g.kv_heads;
  p.group = g.group;
  p.q_stride = g.q_stride;
  p.k_stride = g.k_stride;
  p.v_stride = g.v_stride;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.out = static_cast<const __nv_bfloat16*>(out);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.lse = lse;
  p.q_off = q_offsets;
  p.k_off = kv_offsets;
  p.q_lens = q_lens;
  p.k_lens = kv_lens;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  return launch_cross_bwd(g, p, workspace, static_cast<cudaStream_t>(stream));
}

ress_status ress_cache_plan(const ress_cache_shape* shape, const int32_t* added,
                            const int32_t* lengths, int32_t* table, const int32_t* free_pages,
                            int32_t n_free, const int32_t* cursor, int32_t tokens,
                            int32_t* offsets, int32_t* slots, int32_t* new_lengths,
                            int32_t* new_cursor, void* stream) {
  if (ress_status s = check_pool(shape, false)) return s;
  if (ress_status s = check_table(shape)) return s;
  if (n_free < 0 || tokens < 0) return RESS_ERR_INVALID_ARG;
  if ((int64_t)tokens > kMaxTokens) return RESS_ERR_UNSUPPORTED;   // as attention over them
  if (!added || !lengths || !table || (n_free > 0 && !free_pages) || !cursor || !offsets ||
      (tokens > 0 && !slots) || !new_lengths || !new_cursor)
    return RESS_ERR_INVALID_ARG;
  const void* all[] = {added, lengths, table, free_pages, cursor, offsets, slots, new_lengths,
                       new_cursor};
  for (const void* x : all)
    if (!aligned(x, 4)) return RESS_ERR_INVALID_ARG;
  const void* in[] = {added, lengths, table, free_pages, cursor};
  const void* outs[] = {offsets, slots, new_lengths, new_cursor};
  for (const void* o : outs)
    for (const void* x : in)
      if (o != nullptr && o == x) return RESS_ERR_INVALID_ARG;
  return launch_cache_plan(*shape, added, lengths, table, free_pages, n_free, cursor, tokens,
                           offsets, slots, new_lengths, new_cursor,
                           static_cast<cudaStream_t>(stream));
}

ress_status ress_cache_append(const ress_cache_shape* shape, const void* k, const void* v,
                              int32_t dtype, int64_t k_stride, int64_t v_stride,
                              const int32_t* slots, int32_t tokens, void* k_cache,
                              void* v_cache, float* k_scale, float* v_scale, void* stream) {
  if (ress_status s = check_pool(shape, true)) return s;
  if (dtype != RESS_BF16 && dtype != RESS_F32) return RESS_ERR_INVALID_ARG;
  if (tokens < 0) return RESS_ERR_INVALID_ARG;
  if ((int64_t)tokens > kMaxTokens / 2) return RESS_ERR_UNSUPPORTED;   // bounds the grid
  const int unit = dtype == RESS_F32 ? 4 : 8;
  const int64_t width = (int64_t)shape->kv_heads * kHeadDim;
  const long long ks = row_stride(k_stride, width, unit), vs = row_stride(v_stride, width, unit);
  if (!ks || !vs) return RESS_ERR_INVALID_ARG;
  if (tokens == 0) return RESS_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale)
    return RESS_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return RESS_ERR_INVALID_ARG;
  return launch_cache_append(*shape, k, v, dtype == RESS_F32, ks, vs, slots, tokens, k_cache,
                             v_cache, k_scale, v_scale, static_cast<cudaStream_t>(stream));
}

size_t ress_cache_attn_workspace_bytes(const ress_cache_shape* shape, int32_t heads,
                                       int32_t tokens) {
  if (check_pool(shape, true) != RESS_OK || check_table(shape) != RESS_OK || tokens < 0 ||
      check_heads(heads, shape->kv_heads, shape->head_dim) != RESS_OK)
    return 0;
  return cache_attn_workspace(*shape, heads, tokens);
}

ress_status ress_cache_attn(const ress_cache_shape* shape, int32_t heads, int32_t tokens,
                            const void* q, int64_t q_stride, const void* k_cache,
                            const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* table, const int32_t* lengths,
                            const int32_t* offsets, int32_t step, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (ress_status s = check_pool(shape, true)) return s;
  if (ress_status s = check_table(shape)) return s;
  if (ress_status s = check_heads(heads, shape->kv_heads, shape->head_dim)) return s;
  if (tokens < 0 || step < 0) return RESS_ERR_INVALID_ARG;
  if ((int64_t)tokens > kMaxTokens) return RESS_ERR_UNSUPPORTED;
  const long long qs = row_stride(q_stride, (int64_t)heads * kHeadDim, 8);
  if (!qs) return RESS_ERR_INVALID_ARG;
  if (tokens == 0) return RESS_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !table || !lengths || !offsets || !out)
    return RESS_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(table, 4) ||
      !aligned(lengths, 4) || !aligned(offsets, 4) || !aligned(lse, 4))
    return RESS_ERR_INVALID_ARG;
  if (ress_status s = check_workspace(cache_attn_workspace(*shape, heads, tokens), workspace,
                                      workspace_bytes))
    return s;
  CrossParams p{};
  if ((p.err = device_error_ptr()) == nullptr) return RESS_ERR_CUDA;
  p.nq = tokens;
  p.seqs = shape->requests;
  p.heads = heads;
  p.kv_heads = shape->kv_heads;
  p.group = heads / shape->kv_heads;
  p.q_stride = qs;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_off = offsets;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = table;
  p.lengths = lengths;
  p.pages = shape->pages;
  p.page = shape->page;
  p.max_pages = shape->max_pages;
  p.step = step;
  return launch_cache_attn(p, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
