/*
 * ress.h - C ABI of the B200 (sm_100a) block-sparse global attention library.
 *
 * The library implements the hot path shared by the training-free sparse
 * global-attention methods for multi-view 3D transformers (VGGT-style):
 *
 *   1. ress_select_blocks      pooled block selection: mean-pool Q and K per
 *                              block, per-head softmax over pooled logits,
 *                              optional value-contrast term, exact-budget
 *                              top-k per query block (ties to the lower index).
 *   2. ress_block_sparse_attn  attention restricted to the kept key blocks.
 *   3. ress_block_drift        per-dropped-block drift norm and drop-set drift.
 *
 * ress_select_blocks_cdf is the SparseVGGT variant of stage 1: a per-row
 * cumulative probability threshold instead of a fixed budget.
 *
 * Next to the three stages stand operators for tokens that meet keys of
 * another length: ress_cross_attn and its gradients ress_cross_attn_bwd
 * (packed sequences), and, for views that arrive one after another, a paged
 * key/value cache in 8 bits: ress_cache_plan (block tables and slot maps),
 * ress_cache_append (the writer) and ress_cache_attn (attention over it).
 *
 * Sources: ReSS: Residual-Restoring Sparse Attention for 3D Vision Transformers
 * (thelatestinai.com) - Abstract, Fig. 1, Fig. 3, Table 1, Table S5, Table S6;
 * VASC: Value-Aware Sparse Attention with Cross-Layer Memory (paperlayer.ai) -
 * sections 4.1, 4.2, A.1, A.2, A.3.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are token-major: q, k, v and out are [N][H][d] (d contiguous, one
 *   token row is H*d elements).  lse is [H][N].  idx is [H][nb][budget] int32.
 * - d must be 64.  The block size B (query blocks and key blocks alike) is 64
 *   or 128, and N must be a multiple of B; nb = N / B.  Padding tokens, if
 *   any, are ordinary tokens to the library.
 * - All data pointers are device pointers owned by the caller, on the
 *   current device (the library keeps per-device state, such as its error
 *   flag, and looks it up on the device that is current at the call).
 *   The library never allocates, frees or synchronises; every call is asynchronous and
 *   ordered on `stream` (a cudaStream_t passed as void*, NULL = the legacy
 *   default stream).  Scratch memory comes from the caller's `workspace`,
 *   sized by the matching *_workspace_bytes() query, 256-byte aligned.
 * - Argument checks run on the host before any CUDA call and return
 *   RESS_ERR_INVALID_ARG (bad shape, NULL pointer, budget outside [1, nb],
 *   misaligned pointer), RESS_ERR_UNSUPPORTED (valid but not implemented,
 *   e.g. d != 64) or RESS_ERR_WORKSPACE (workspace too small).  A failed
 *   launch returns RESS_ERR_CUDA.  When N == 0 the call returns RESS_OK and
 *   launches nothing.
 * - Kernels never trap.  A device-side wait that exceeds its time limit, or a
 *   kept-block index outside [0, nb) found in a caller-provided idx (such an
 *   index is skipped), sets a device error flag that ress_check_device_errors()
 *   reports and clears.
 */
#ifndef RESS_H
#define RESS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  RESS_OK = 0,
  RESS_ERR_INVALID_ARG = 1,
  RESS_ERR_UNSUPPORTED = 2,
  RESS_ERR_WORKSPACE = 3,
  RESS_ERR_CUDA = 4,
  RESS_ERR_TIMEOUT = 5,
  RESS_ERR_BAD_INDEX = 6
} ress_status;

typedef enum {
  RESS_BF16 = 0, /* bfloat16 q, k, v (and out) */
  RESS_F32 = 1   /* float32 q, k, v (and out); attention and drift stage them to bf16 */
} ress_dtype;

typedef struct {
  int64_t n;        /* N: tokens of all views concatenated (multiple of block) */
  int32_t heads;    /* H: attention heads, 1..64 */
  int32_t head_dim; /* d: must be 64 */
  int32_t block;    /* B: 64 or 128 */
  int32_t dtype;    /* ress_dtype of q, k and v */
} ress_shape;

/*
 * Per-view layout of the concatenated sequence, for the layout-aware entry
 * points (VASC 4.2 and A.5: camera and register queries keep dense
 * attention, key blocks made only of special tokens are always kept, and
 * padding takes no part in pooling or attention).  Every view occupies
 * tokens_per_view consecutive tokens; its positions 0 .. real_tokens - 1
 * carry data and the rest is padding; positions 0 .. special_tokens - 1 are
 * the special (camera, register) tokens.  Requirements: tokens_per_view a
 * multiple of the block size and a divisor of N, 1 <= real_tokens <=
 * tokens_per_view, 0 <= special_tokens <= real_tokens.  A VGGT view is
 * {1408, 1374, 5}: 1 camera + 4 register + 37 x 37 patch tokens, padded to
 * 22 blocks of 64.
 */
typedef struct {
  int32_t tokens_per_view;
  int32_t real_tokens;
  int32_t special_tokens;
} ress_layout;

/* Library version, (major << 16) | minor. */
int ress_version(void);

/* Human-readable name of a status code; never NULL. */
const char* ress_status_string(ress_status status);

/*
 * Workspace bytes that ress_select_blocks needs for `shape` and `lambda`
 * (0 if the shape is invalid).  Layout, each array 256-byte aligned, with
 * nb_pad = nb rounded up to 256:
 *   - lambda == 0, budget < nb <= 2304 (the tensor-core selection):
 *     Qbar [H][nb][64] f32, then the pooled keys split into tf32 high and low
 *     parts Khi, Klo [H][nb_pad][64] f32, the high parts of 128 evenly spaced
 *     sample keys [H][128][64], the key norms [H][nb] f32, one int32 count
 *     (in a 256-byte slot) and a row list [H][nb] int32;
 *   - otherwise (and for ress_select_blocks_cdf): Qbar [H][nb][64],
 *     Kbar^T [H][64][nb_pad], then Vbar [H][nb][64] and contrast [H][nb]
 *     when lambda > 0, all float32.
 * The size returned covers both layouts when lambda == 0.
 */
size_t ress_select_workspace_bytes(const ress_shape* shape, float lambda);

/*
 * Stage 1: pooled block selection (ReSS Table S5, SpargeAttn row: pooled
 * query/key inner products; VASC 4.1: pooled relevance plus neighbouring
 * value contrast; VASC A.2: an exact-capacity binary Top-K mask).
 *
 * For each head h and query block i:
 *   Qbar_i = mean of the B query tokens of block i (same for Kbar_j, Vbar_j),
 *   s_ij   = (Qbar_i . Kbar_j) / sqrt(d),
 *   p_ij   = softmax over all nb key blocks j of s_ij,
 *   c_j    = ||Vbar_j - Vbar_{j-1}||_2 for j >= 1, c_0 = 0,
 *   score  = p_ij + lambda * c_j,
 * and idx[h][i][0..budget) receives the `budget` blocks of largest score in
 * ascending block order; equal scores go to the lower block index.  With
 * lambda == 0 the ranking uses s_ij, which orders the row as p_ij does.
 *
 *   q, k    [N][H][64] of shape->dtype, 16-byte aligned.
 *   v       [N][H][64], read only when lambda > 0 (may be NULL otherwise).
 *   budget  kept key blocks per query block, 1 <= budget <= nb.
 *   lambda  contrast weight, finite and >= 0.
 *   idx     out, [H][nb][budget] int32.
 *   Supported sizes: nb <= 4096.
 */
ress_status ress_select_blocks(const ress_shape* shape, const void* q, const void* k,
                               const void* v, int32_t budget, float lambda, int32_t* idx,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stage 1 for callers that cannot allocate device memory.  The pages have no
 * counterpart to this entry point; it exists for callers that may not call
 * cudaMalloc or hold a workspace of their own (for example a plugin running
 * inside another framework's allocator, or a loop in which an allocation,
 * which can synchronise the device, is not allowed).
 *
 * Same arguments, checks and result as ress_select_blocks, without the
 * workspace: the scratch lives in one fixed 32 MiB array in device memory
 * that the library owns (H = 16 and nb <= 2,200 fit, with the value
 * contrast).  Every GPU that loads the library holds that array until the
 * process exits.  A problem whose ress_select_workspace_bytes() exceeds
 * 32 MiB is rejected with RESS_ERR_WORKSPACE before anything is launched.
 *
 * - The first call on a device looks up the array's device address (one
 *   cudaGetSymbolAddress with that device current); make that first call
 *   before any stream capture.  The call allocates nothing.
 * - All calls share the one array, and each call overwrites every scratch
 *   value it reads, so nothing needs to start at zero.  Calls that overlap on
 *   the GPU (different streams, or different host threads, on one device)
 *   race on the array and must be ordered by the caller.
 */
ress_status ress_select_blocks_noalloc(const ress_shape* shape, const void* q, const void* k,
                                       const void* v, int32_t budget, float lambda,
                                       int32_t* idx, void* stream);

/*
 * Stage 1 with the cumulative (CDF) threshold of SparseVGGT instead of a fixed
 * budget (ReSS Table S5: with the similarity gate off, selection is a
 * cumulative threshold on pooled query/key inner products; ReSS Table 2, row
 * "+ CDF threshold").  For each head h and query block i, with p_ij the pooled
 * probabilities of ress_select_blocks (lambda = 0), the count is the smallest
 * m >= 1 such that the m blocks of largest p (equal values in index order) sum
 * to at least tau, or nb if the total never reaches tau.
 *
 *   q, k       as for ress_select_blocks (no V: the rule has no contrast term).
 *   tau        0 < tau <= 1.
 *   capacity   1 <= capacity <= nb: the length of every idx row.
 *   counts     out, [H][nb] int32: the count of every row (it may exceed
 *              capacity).
 *   idx        out, [H][nb][capacity] int32: the top min(count, capacity)
 *              blocks of the row in ascending order, then the last of them
 *              repeated to the end of the row, so that idx with
 *              budget = capacity is a valid kept list for
 *              ress_block_sparse_attn (duplicates count once there).
 *   workspace  ress_select_workspace_bytes(shape, 0) bytes, 256-byte aligned.
 *   Supported sizes: nb <= 4096.
 *   The probabilities are float32 and their running sum is exact (fixed point
 *   in units of 2^-40, independent of the summation order), so the result is
 *   deterministic, and a count can differ from an evaluation in float64 only
 *   where the cumulative mass lies within about 1e-6 of tau.
 */
ress_status ress_select_blocks_cdf(const ress_shape* shape, const void* q, const void* k,
                                   float tau, int32_t capacity, int32_t* counts, int32_t* idx,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stage 1 with a per-view layout (VASC 4.2 and A.5).  As ress_select_blocks
 * with lambda = 0, except that a block's pooled mean is over its valid
 * (non-padding) tokens only, a key block without a valid token (it pools to
 * zero) ranks below every other block, and a key block whose valid tokens are
 * all special ranks above every other block (such blocks are kept first,
 * lowest index first if there are more of them than the budget).
 *
 *   layout     as described at ress_layout.
 *   workspace  ress_select_workspace_bytes(shape, 0) bytes.
 */
ress_status ress_select_blocks_layout(const ress_shape* shape, const ress_layout* layout,
                                      const void* q, const void* k, int32_t budget,
                                      int32_t* idx, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Workspace bytes of ress_select_blocks_restore (0 if the shape is invalid):
 * Qbar [H][nb][64], Kbar^T [H][64][nb_pad] and Vbar^T [H][64][nb_pad],
 * float32, each 256-byte aligned.
 */
size_t ress_restore_workspace_bytes(const ress_shape* shape);

/*
 * Stage 1 by drift with iterative residual restoration (ReSS Abstract, Fig. 1,
 * Fig. 3(b)-(c), Fig. 7, Table S3), on pooled contributions.  For query block
 * i of head h, key block j contributes c_j = p_ij Vbar_j to the pooled output
 * (p_ij the pooled probabilities of ress_select_blocks).  The drift score is
 * |c_j|; the initial kept set is the `budget` blocks of largest score (ties
 * to the lower index).  Each of up to `rounds` restoration rounds takes the
 * drop set D and T = sum_{j in D} c_j, forms the pairs of the `candidates`
 * dropped blocks of largest 2 <T, c_b> - |c_b|^2 and the `candidates` kept
 * blocks of smallest 2 <T, c_a> + |c_a|^2 (ties to the lower index), and swaps
 * the pair of smallest |T - c_b + c_a| (ties: lower b, then lower a) when
 * that is below |T|; otherwise restoration stops.  The swap rule and the
 * pooled contributions are this library's reading: the pages give neither.
 *
 *   rounds       0 .. 64 (0: the initial set).
 *   candidates   1 .. 16 per side.
 *   idx          out, [H][nb][budget] int32, ascending.
 *   drift_init   out, [H][nb] float32, |sum over the initial drop set|; or NULL.
 *   drift_final  out, [H][nb] float32, the same for the result; or NULL.
 *   Supported sizes: nb <= 4096.  Arithmetic in float32; a decision between
 *   two values equal to float32 rounding may go either way.
 */
ress_status ress_select_blocks_restore(const ress_shape* shape, const void* q, const void* k,
                                       const void* v, int32_t budget, int32_t rounds,
                                       int32_t candidates, int32_t* idx, float* drift_init,
                                       float* drift_final, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of ress_select_blocks_vasc (0 if the shape is invalid):
 * Qbar [H][nb][64], Kbar^T and Vbar^T [H][64][nb_pad] float32, then per pair
 * the contrast and the memory's ranking copy (float32), the demand sum
 * (uint64) and the service count (uint32), [H][(nb + 1) / 2] each; every
 * array 256-byte aligned.
 */
size_t ress_vasc_workspace_bytes(const ress_shape* shape);

/*
 * Stage 1 as VASC selects it, one global layer per call: value-aware demand,
 * a binary mask of exactly c_h blocks per row, and the cross-layer memory
 * settled by what was executed (VASC 4.1, 4.2, 4.3, A.1 - A.5; per-head
 * budgets c_h as in ReSS Fig. 3 and Table 2).
 *
 * Key blocks form fixed pairs of neighbours (2p, 2p+1), p < (nb + 1) / 2; an
 * odd final block is a singleton.  For head h and query block i, with p_ij
 * the pooled probabilities of ress_select_blocks:
 *   rho_p  = sqrt( (1/64) sum_d (Vbar_2p,d - Vbar_2p+1,d)^2 ), 0 for a
 *            singleton (the RMS contrast of the pair); 1 for every pair when
 *            value_aware == 0 (the contrast set to one);
 *   a_ij   = min(1, c_h * p_ij rho_pair(j) / sum_j p_ij rho_pair(j))
 *            (0 when the sum is 0): the demand, rescaled to the capacity and
 *            clipped at one;
 *   mhat_p = memory_p / max over the head's pairs (0 when that is 0): the
 *            ranking copy of the memory;
 *   kept   = the c_h largest a_ij + mhat_pair(j), ties to the lower index.
 * Then, with D_p and S_p the means of a_ij and of the kept mask over all query
 * blocks i and the children j of pair p,
 *   memory_p <- max(0, memory_p + D_p - S_p).
 * How the contrast modulates the relevance (a factor), how memory enters the
 * ranking (added), how it is normalised (by the head's largest balance) and
 * the rescaling (proportional, one clip) are this library's readings.
 *
 *   v            [N][H][64], needed when value_aware != 0 (else may be NULL).
 *   budgets      HOST array of H int32: c_h, 1 <= c_h <= capacity.
 *   capacity     1 <= capacity <= nb: the length of every idx row.
 *   value_aware  1: contrast on; 0: contrast one.
 *   reset        1: the memory is taken as zero on entry (the first global
 *                layer of an inference, or a changed layout); 0: carried in.
 *   memory       in/out, device [H][(nb + 1) / 2] float32 (>= 0).
 *   idx          out, [H][nb][capacity] int32: row (h, i) holds its c_h kept
 *                blocks ascending, then the last of them repeated, a valid
 *                kept list for ress_block_sparse_attn with budget = capacity.
 *   demand       out, [H][(nb + 1) / 2] float32, D; or NULL.
 *   service      out, [H][(nb + 1) / 2] float32, S; or NULL.
 *   workspace    ress_vasc_workspace_bytes(shape) bytes, 256-byte aligned.
 *   Supported sizes: nb <= 4096.  The demand sums are exact in fixed point
 *   (units of 2^-32), so memory, demand and service do not depend on the
 *   order of the kernel's blocks; the scores are float32, so a ranking
 *   decision between two values equal to float32 rounding may go either way.
 */
ress_status ress_select_blocks_vasc(const ress_shape* shape, const void* q, const void* k,
                                    const void* v, const int32_t* budgets, int32_t capacity,
                                    int32_t value_aware, int32_t reset, float* memory,
                                    int32_t* idx, float* demand, float* service,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Workspace bytes that ress_block_sparse_attn and ress_block_drift need:
 * 0 for bf16 inputs; 3 * N * H * 64 * 2 for float32 inputs (bf16 copies of
 * q, k and v).
 */
size_t ress_attn_workspace_bytes(const ress_shape* shape);

/*
 * Stage 2: block-sparse attention forward (ReSS Table S6: the selection feeds
 * one shared block-sparse kernel on the block grid; VASC 4.2: the binary mask
 * is passed directly to the sparse kernel; ReSS Table S5: bidirectional, no
 * causal mask).
 *
 * For query token n of block i and head h, with kept set K(h, i) = idx[h][i]:
 *   out[n][h] = sum_{t in K} softmax_t((q[n][h] . k[t][h]) / sqrt(d)) v[t][h],
 * normalised over the kept tokens only, and
 *   lse[h][n] = ln sum_{t in K} exp((q[n][h] . k[t][h]) / sqrt(d)).
 *
 *   idx    [H][nb][budget] int32 device array; rows need not be sorted or
 *          unique (duplicates count once); entries outside [0, nb) are skipped
 *          and flagged (RESS_ERR_BAD_INDEX via ress_check_device_errors).
 *   out        [N][H][64] of `out_dtype` (RESS_BF16 or RESS_F32, independent
 *              of the input dtype).
 *   lse        [H][N] float32, or NULL.
 *   Supported sizes: nb <= 10,000 (the kept-block lists live in shared
 *   memory); larger grids return RESS_ERR_UNSUPPORTED.
 *   The contractions run on bf16 operands with float32 accumulation; the
 *   probabilities enter P V as bf16 and the row normaliser is the sum of those
 *   same bf16 values, so each output row is a convex combination of kept
 *   values, and lse is the log of that same sum (it differs from the float32
 *   log-sum-exp by at most ln(1 + 2^-9) < 2e-3).
 */
ress_status ress_block_sparse_attn(const ress_shape* shape, const void* q, const void* k,
                                   const void* v, int32_t budget, const int32_t* idx,
                                   void* out, int32_t out_dtype, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of ress_block_sparse_attn_layout: the float32 staging of
 * ress_attn_workspace_bytes (float32 inputs only), then the special rows'
 * gathered queries, outputs and lse (0 bytes when special_tokens == 0).
 * out_dtype as for the call.  0 if the shape or layout is invalid.
 */
size_t ress_attn_layout_workspace_bytes(const ress_shape* shape, const ress_layout* layout,
                                        int32_t out_dtype);

/*
 * Stage 2 with a per-view layout (VASC 4.2 and A.5).  As
 * ress_block_sparse_attn, except that
 *   - padding keys never enter a softmax;
 *   - a padding query row writes 0 and lse -inf (so does a row whose kept
 *     blocks hold no valid key);
 *   - a special query (the first special_tokens tokens of each view) attends
 *     densely to every valid key of the sequence, whatever idx says.
 *   workspace  ress_attn_layout_workspace_bytes(shape, layout, out_dtype)
 *              bytes, 256-byte aligned (NULL when that is 0).
 */
ress_status ress_block_sparse_attn_layout(const ress_shape* shape, const ress_layout* layout,
                                          const void* q, const void* k, const void* v,
                                          int32_t budget, const int32_t* idx, void* out,
                                          int32_t out_dtype, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * Stage 3: drift of the dropped blocks (ReSS Abstract and Fig. 3: the drift
 * score measures how much masking a block shifts what attention writes into
 * the residual stream; the drift of a drop set depends on the directions of
 * the contributions, Fig. 9 plots quality against it).
 *
 * For query block i of head h and every dropped block j (not in idx[h][i]),
 * in ascending j order r = 0 .. nb - budget - 1:
 *   C_j[n][:] = sum_{t in block j} exp((q[n] . k[t]) / sqrt(d) - lse[h][n]) v[t][:]
 *   drift[h][i][r] = ||C_j||_F over the B x 64 matrix,
 *   set_drift[h][i] = || sum_{j dropped} C_j ||_F.
 * lse is the kept-set normaliser written by ress_block_sparse_attn for the
 * same idx.
 *
 *   idx        as for ress_block_sparse_attn, but rows must hold `budget`
 *              distinct in-range blocks (the drift row length is nb - budget).
 *              A row that names a block twice is flagged (RESS_ERR_BAD_INDEX,
 *              detail 5, via ress_check_device_errors); the drift entries
 *              such a row would place beyond nb - budget are not written.
 *   lse        [H][N] float32 from ress_block_sparse_attn.
 *   drift      out, [H][nb][nb - budget] float32 (may be NULL when budget == nb).
 *   set_drift  out, [H][nb] float32, or NULL.
 */
ress_status ress_block_drift(const ress_shape* shape, const void* q, const void* k,
                             const void* v, int32_t budget, const int32_t* idx,
                             const float* lse, float* drift, float* set_drift,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Debug aid: checks a kept-block list on the device, ordered on `stream`
 * (VASC A.2: the binary Top-K mask has exact capacity, so a row names
 * `budget` distinct blocks; ress_select_blocks writes them ascending).
 * Launches one small kernel that reads idx and writes nothing but the device
 * error flag: RESS_ERR_BAD_INDEX, reported by ress_check_device_errors with
 * detail 80 (an entry outside [0, nb)), 81 (a row repeats a block in
 * adjacent positions) or 82 (a row not in ascending order).  The first error
 * found wins.
 *
 *   idx      [H][nb][budget] int32 device array, 4-byte aligned.
 *   budget   1 <= budget <= nb.
 */
ress_status ress_validate_idx(const ress_shape* shape, int32_t budget, const int32_t* idx,
                              void* stream);

/*
 * Stage 3 with a per-view layout (VASC 4.2 and A.5).  As ress_block_drift,
 * except that only valid keys enter a contribution and only the valid,
 * non-special queries count: the rows of padding and special queries (which
 * attend densely and drop nothing) of every C_j are zero.  lse comes from
 * ress_block_sparse_attn_layout with the same idx.
 */
ress_status ress_block_drift_layout(const ress_shape* shape, const ress_layout* layout,
                                    const void* q, const void* k, const void* v, int32_t budget,
                                    const int32_t* idx, const float* lse, float* drift,
                                    float* set_drift, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * Shape of ress_cross_attn and ress_cross_attn_bwd: packed sequences of
 * query tokens and of key tokens, which need not be equally long.
 *
 * q, out, dout, dq are [nq][heads][64], k, v, dk, dv are [nk][kv_heads][64];
 * query head h reads key head h / (heads / kv_heads).  A token row of q, k or
 * v may be part of a wider row (a slice of a fused projection): q_stride,
 * k_stride and v_stride are the elements from one token row to the next, a
 * multiple of 8 and at least the row's own heads * 64; 0 stands for exactly
 * that.  Every other tensor is dense.
 *
 * Sequence b is the query rows q_offsets[b] .. q_offsets[b + 1] - 1 and the
 * key rows kv_offsets[b] .. kv_offsets[b + 1] - 1 (int32 device arrays of
 * seqs + 1 entries; both NULL with seqs == 1: all rows).  q_lens and kv_lens
 * (int32 device arrays of seqs entries, or NULL) mark padding: only the first
 * q_lens[b] / kv_lens[b] rows of a sequence carry data.  Padding keys enter
 * no softmax and are never used as numbers (they may hold NaN); a padding
 * query row writes 0 and lse -inf, and so does a query whose sequence has no
 * key.  Rows of no sequence (before the first offset, behind the last) are
 * left as they were in every output.
 *
 * The arrays live on the device, so the kernels check them: a sequence whose
 * offsets are out of range or decrease is taken as empty and flagged
 * (RESS_ERR_BAD_INDEX, detail 90 for queries, 91 for keys), a length outside
 * its sequence is clamped to it and flagged (92, 93).
 *
 * dtype must be RESS_BF16: the contractions take bf16 operands, and a float32
 * input would be rounded to them unseen.  1 <= heads <= 64, kv_heads divides
 * heads, 1 <= seqs <= 8192, nq and nk up to 2^30.
 */
typedef struct {
  int64_t nq;
  int64_t nk;
  int32_t seqs;
  int32_t heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t dtype;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
} ress_cross_shape;

/* Workspace bytes of ress_cross_attn / ress_cross_attn_bwd (0: none needed or
 * the shape is invalid): partial sums where a long key (or query) range is
 * split over several CTAs, and for the gradients delta [heads][nq] float32. */
size_t ress_cross_workspace_bytes(const ress_cross_shape* shape);
size_t ress_cross_bwd_workspace_bytes(const ress_cross_shape* shape);

/*
 * Attention of one set of tokens over another (dense, bidirectional): for
 * query row i of sequence b and head h, over the keys t of sequence b,
 *   out[i][h] = sum_t softmax_t((q[i][h] . k[t][h']) / sqrt(d)) v[t][h'],
 *   lse[h][i] = ln sum_t exp((q[i][h] . k[t][h']) / sqrt(d)).
 * Every other entry point of this library attends a sequence to itself; this
 * one serves queries that are not among the keys (a new view against stored
 * ones, a decoder's tokens against the encoded views).
 *
 *   out        [nq][heads][64] bf16;  lse  [heads][nq] float32, or NULL.
 *   workspace  ress_cross_workspace_bytes(shape) bytes, 256-byte aligned
 *              (NULL when that is 0).
 *   Contractions on bf16 operands with float32 accumulation; probabilities
 *   enter P V as bf16, their sum and lse are float32 sums of the unrounded
 *   ones.  Results do not depend on the run: no atomics add numbers.  Outputs
 *   must not overlap inputs.
 *   Logits are made for magnitudes up to 2^30.  Beyond, where float32 keeps them
 *   to 64 at best, a row may come out as NaN, since the difference from the row's
 *   maximum holds what rounding took from the maximum.  (A kernel without that
 *   limit was built; it cost every call 5 %.)
 */
ress_status ress_cross_attn(const ress_cross_shape* shape, const void* q, const void* k,
                            const void* v, const int32_t* q_offsets, const int32_t* kv_offsets,
                            const int32_t* q_lens, const int32_t* kv_lens, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of ress_cross_attn.  With P = exp(S - lse), S = q . k / sqrt(d),
 * delta[i] = dout[i] . out[i] and dS = P (dout . v - delta):
 *   dq[i] = sum_t dS[i][t] k[t] / sqrt(d),
 *   dk[t] = sum_i dS[i][t] q[i] / sqrt(d),   dv[t] = sum_i P[i][t] dout[i],
 * where dk and dv also add over the heads / kv_heads query heads that share a
 * key head.  Rows without a partner (no key, no query) and padding rows get
 * 0; rows of no sequence are left as they were.
 *
 *   out, lse   as ress_cross_attn wrote them (an lse of -inf marks a row
 *              without a key).
 *   dout       [nq][heads][64] bf16.
 *   dq         [nq][heads][64] bf16; dk, dv [nk][kv_heads][64] bf16.
 *   workspace  ress_cross_bwd_workspace_bytes(shape) bytes, 256-byte aligned.
 *   P = exp(S - lse) takes lse as float32, so it is off by 2^-24 |lse|: gradients
 *   mean something for logits up to about 2^16.
 *   dS enters dq as two bf16 numbers (16 bits); P enters dv, and dS dk, as one for
 *   sequences of more than 128 keys and as two for shorter ones.  All sums are
 *   float32 in a fixed order.
 */
ress_status ress_cross_attn_bwd(const ress_cross_shape* shape, const void* q, const void* k,
                                const void* v, const void* out, const float* lse,
                                const void* dout, const int32_t* q_offsets,
                                const int32_t* kv_offsets, const int32_t* q_lens,
                                const int32_t* kv_lens, void* dq, void* dk, void* dv,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * A paged key/value cache in 8 bits for views that arrive one after another.
 *
 * The pool holds `pages` pages of `page` tokens (64 or 128, the library's
 * blocks).  k_cache and v_cache are [pages][kv_heads][page][64] e4m3 codes
 * (one byte each); k_scale and v_scale are [pages][kv_heads] float32: a page
 * and head stands for code * scale.  A scale is a power of two: e4m3 has a
 * binary exponent of its own, so a finer scale would buy no precision, while
 * a power of two divides and multiplies exactly, and a scale that grows
 * re-codes older tokens without rounding them again, except where they fall
 * among e4m3's smallest (subnormal) numbers.  Request r keeps its tokens 0 ..
 * lengths[r] - 1 in the pages table[r][0], table[r][1], ... ([requests]
 * [max_pages] int32; entries behind the last page in use are not read).
 */
typedef struct {
  int32_t pages;      /* pages of the pool */
  int32_t page;       /* tokens per page: 64 or 128; pages * page < 2^31 */
  int32_t kv_heads;   /* 1..64 */
  int32_t head_dim;   /* must be 64 */
  int32_t requests;   /* rows of the table, 1..8192 */
  int32_t max_pages;  /* entries per table row; max_pages * page < 2^31 */
} ress_cache_shape;

/*
 * Block tables and slot maps for the tokens that every request adds.
 *
 * Request r holds lengths[r] tokens and adds added[r].  It needs
 * ceil((lengths[r] + added[r]) / page) - ceil(lengths[r] / page) new pages;
 * these are taken in request order from free_pages, starting at entry
 * cursor[0], and written behind the row's pages in use:
 *   table[r][ceil(lengths[r] / page) + i] = free_pages[cursor + need_0 + ... + need_(r-1) + i].
 * The added tokens are packed in request order: those of r are offsets[r] ..
 * offsets[r + 1] - 1, and token t of them goes to cell
 *   slots[t] = table[r][pos / page] * page + pos % page,  pos = lengths[r] + t - offsets[r].
 *
 * A request that does not fit (its row too short, the free list used up
 * before or in it, more tokens than the slot map holds, a negative length or
 * count) is left as it is: its length stays, its tokens get slot -1, no page
 * is taken for it, and the device error RESS_ERR_BAD_INDEX is flagged (detail
 * 100 row or counts, 101 free list, 102 slot map).  Once the free list or the
 * slot map is used up, later requests that need of it fail too.  A page id
 * outside the pool, in the free list or the table, gives its tokens slot -1
 * and is flagged (103).
 *
 *   added, lengths  [requests] int32;  table in/out;  free_pages [n_free] int32.
 *   cursor          [1] int32: first entry of free_pages not yet taken.
 *   offsets         out, [requests + 1] int32.
 *   slots           out, [tokens] int32, tokens up to 2^30; entries behind the added
 *                   tokens get -1.
 *   new_lengths     out, [requests] int32;  new_cursor  out, [1] int32.
 *   The outputs other than table must not overlap the inputs (every CTA reads
 *   the inputs while others write), which the call checks for equal pointers.
 *   shape->kv_heads and head_dim are not used.  One launch, no workspace.
 */
ress_status ress_cache_plan(const ress_cache_shape* shape, const int32_t* added,
                            const int32_t* lengths, int32_t* table, const int32_t* free_pages,
                            int32_t n_free, const int32_t* cursor, int32_t tokens,
                            int32_t* offsets, int32_t* slots, int32_t* new_lengths,
                            int32_t* new_cursor, void* stream);

/*
 * Writes new tokens into the cache: token t (row t of k and v, [tokens]
 * [kv_heads][64] of `dtype`, bf16 or float32, row strides as in
 * ress_cross_shape) goes to cell slots[t]; a negative slot skips the token.
 *
 * Slots of one page must stand together and ascend by one (as
 * ress_cache_plan writes them): a run.  For each run, head and tensor, with c
 * the run's first cell and amax the largest |x| of its tokens,
 *   s = smallest power of two >= 2^-100 with amax <= 448 s, at most 2^119,
 *   s = max(s, old scale) when c > 0;
 * the page's scale becomes s, the run's codes are x / s rounded to e4m3
 * (nearest, ties to even), and when c > 0 the codes of cells 0 .. c - 1 are
 * re-coded to the new scale.  A run that starts at cell 0 takes the page over:
 * an older scale is forgotten.  Cells behind the run keep their codes.
 *
 *   A page that appears in two runs of one call gets an undefined content
 *   (two runs write it at once); slots outside the pool are skipped and
 *   flagged (RESS_ERR_BAD_INDEX, detail 104).  Values must be at most 448 * 2^119
 *   (2.98e38) in magnitude: one that is not is flagged (RESS_ERR_INVALID_ARG,
 *   detail 105).  Its code is the largest number, or NaN for NaN; infinities and
 *   NaN do not count for the scale.
 *   The scale of a page that is continued must be one that an append wrote.
 *   tokens may be up to 2^29.  shape->requests and max_pages are not used.  One
 *   launch, no workspace.
 */
ress_status ress_cache_append(const ress_cache_shape* shape, const void* k, const void* v,
                              int32_t dtype, int64_t k_stride, int64_t v_stride,
                              const int32_t* slots, int32_t tokens, void* k_cache,
                              void* v_cache, float* k_scale, float* v_scale, void* stream);

/*
 * Workspace bytes of ress_cache_attn (0 if the shape is invalid): partial
 * rows of requests whose keys are split over several CTAs.
 */
size_t ress_cache_attn_workspace_bytes(const ress_cache_shape* shape, int32_t heads,
                                       int32_t tokens);

/*
 * Attention of new tokens over the cache.  The queries of request r are the
 * rows offsets[r] .. offsets[r + 1] - 1 of q ([tokens][heads][64] bf16, row
 * stride q_stride elements, 0 = dense), the last of the request's lengths[r]
 * tokens (which have been appended): row i of n stands at position
 * lengths[r] - n + i.  Query head h reads key head h / (heads / kv_heads).
 *   out[t][h] = sum_u softmax_u((q . K_u) / sqrt(d)) V_u,  lse[h][t] the log-sum-exp,
 * over the cached tokens u < end(t):
 *   step == 0   end = lengths[r]: every token sees every other;
 *   step >= 1   end = min(lengths[r], (position / step + 1) * step): a token
 *               sees its own group of `step` tokens and the earlier ones
 *               (step 1: causal; step = tokens of a view: views in order).
 * A row that sees nothing (an empty request; with a step, a position before 0)
 * writes 0 and lse -inf.  Rows of no request are left as they were.
 *
 *   table     [requests][max_pages] int32, lengths [requests] int32, offsets
 *             [requests + 1] int32.  Flagged as RESS_ERR_BAD_INDEX: offsets
 *             out of range or descending (detail 90; the request is taken as
 *             empty), a length outside 0 .. max_pages * page (94; clamped), a
 *             page outside the pool (95; its keys are left out).  Scales must be
 *             powers of two from 2^-100 to 2^119, or zero; a page with another one
 *             is flagged (RESS_ERR_INVALID_ARG, detail 96) and its keys are left out.
 *   out       [tokens][heads][64] bf16;  lse [heads][tokens] float32 or NULL.
 *   workspace ress_cache_attn_workspace_bytes() bytes, 256-byte aligned.
 *   Codes and queries are multiplied exactly; probabilities enter P V as
 *   bf16 or f16, their sums and lse are float32.  Cells behind lengths[r] are
 *   never used as numbers.  A token before them whose key or value holds a NaN
 *   code (the append that made it was flagged) makes NaN every row that sees it,
 *   all 64 values and lse, and changes no other row.  Logits up to 2^30, as in
 *   ress_cross_attn.
 *   tokens may be up to 2^30.  Which of two kernels serves the call is chosen from
 *   the average query rows per request: requests that add whole views and requests
 *   that add a token each are faster in two calls (by about half).  The kernel for
 *   few rows reads all of a request's keys whatever the step.
 */
ress_status ress_cache_attn(const ress_cache_shape* shape, int32_t heads, int32_t tokens,
                            const void* q, int64_t q_stride, const void* k_cache,
                            const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* table, const int32_t* lengths,
                            const int32_t* offsets, int32_t step, void* out, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, then reports and clears the device error flag that
 * the kernels set: RESS_ERR_TIMEOUT (a device wait ran out of time),
 * RESS_ERR_BAD_INDEX (an idx entry outside [0, nb) was skipped, or what the entry
 * points above say), RESS_ERR_INVALID_ARG (a value or a scale that the cache does
 * not take), RESS_OK if none, RESS_ERR_CUDA if the synchronisation itself failed.  `detail`, if not
 * NULL, receives a kernel-specific code of the first error (0 if none).
 */
ress_status ress_check_device_errors(void* stream, int32_t* detail);

/*
 * Name and message of the last CUDA error behind a RESS_ERR_CUDA returned to
 * the calling host thread ("" if none).  The string stays valid until the
 * thread's next library call.
 */
const char* ress_last_cuda_error(void);

/*
 * Test hook: y[i] = 2^x[i] computed by the polynomial exponential that the
 * attention kernel uses for part of its probabilities (range reduction plus
 * a degree-3 minimax polynomial on the FMA pipe; relative error <= 1e-4 for
 * -100 <= x <= 8, a finite value below 2^-99 under that).  x and y are device
 * arrays of n float32.
 */
ress_status ress_test_exp2(const float* x, float* y, int32_t n, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RESS_H */
