/*
 * moe_tokens.h -- C ABI of the operators around the experts' products: tokens sorted by expert and
 * back with the router's weights, and low-rank adapters of many requests (or of many experts) beside
 * a shared projection, each with its gradient (library: expert_offload_lru_amd/libmoe_offload.so).
 *
 * moe_layer_forward (moe_offload.h) does its own grouping; these entry points are for products that
 * a caller runs on the routed rows itself: adapters trained or served beside the frozen 4-bit
 * experts, or experts of its own.  The gradients are of these operators alone: the layer's experts
 * and router have none.  The layer gives its routing as host arrays (moe_cache_last_routing), so a
 * step that takes ids and gates from there copies them to the device, and no one graph holds both.
 *
 * Conventions (those of moe_offload.h, and)
 *  - Every function enqueues its kernels on `stream` (a hipStream_t as void*) of the current device
 *    and returns; it waits for nothing, allocates nothing and records nothing but kernels, so any
 *    call may be captured into a graph.  Pointers are memory of that device.
 *  - Two calls may run at once if neither writes what the other reads or writes (workspaces included).
 *  - dtype (MOE_T_*) is the type of every tensor without a type of its own; gates, scales and the
 *    adapters' gradients are fp32, indexes int32.  Sums (and the adapters' v and u below) are held
 *    in fp32, and a result is rounded once.  An infinite operand gives the infinities and NaN that
 *    the formula gives.
 *  - Matrices are row-major; ld is the number of elements from one row to the next (>= the row's
 *    length).  No alignment beyond the element's own is needed; rows that start at multiples of 16
 *    bytes are the fast case.
 *  - An output may not overlap an input or another output, but out may be base (the same pointer and
 *    ld), and d_x may be dx_base.  A matrix is taken as all from its first to its last element: two
 *    column ranges of one wider matrix overlap.
 *  - Errors: MOE_ERR_INVALID (a NULL or overlapping tensor, a size or ld out of range, an unknown
 *    type, a workspace that is too small), MOE_ERR_UNSUPPORTED (a size
 *    over the limits stated), both before anything is enqueued, and MOE_ERR_HIP (a launch failed; the
 *    kernels before it may run).
 *  - Index values are checked on the device: one out of range counts as "none".
 *  - Results do not depend on timing: the same inputs give the same bits.
 */
#ifndef MOE_TOKENS_H
#define MOE_TOKENS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- element types */
#define MOE_T_F32   0
#define MOE_T_F16   1
#define MOE_T_BF16  2

/* Tokens sorted by expert.  ids [n_tokens x top_k]: the picked experts; a value outside
 * 0 .. n_experts-1 (-1, say) is no pick, and a token may pick an expert twice.  The valid picks
 * p = t*top_k + j, in the order of (ids[p], p), become rows 0 .. R-1:
 *   offsets [n_experts + 1]       rows of expert e: offsets[e] .. offsets[e+1]; offsets[n_experts] = R
 *   pos     [n_tokens x top_k]    row of a pick, -1 for no pick
 *   src     [n_tokens * top_k]    pick of a row, -1 from R on
 *   expert  [n_tokens * top_k]    expert of a row, -1 from R on
 *   rows    [n_tokens*top_k x hidden]   rows[pos[p]] = x[p / top_k]; left as they were from R on
 * x and rows may both be NULL (hidden and the ld are then ignored): only the order is made.
 * n_tokens = 0 writes offsets alone.  workspace: moe_tokens_workspace bytes (NULL if that is 0),
 * 4-byte aligned; it holds nothing between calls.  Limits here and below: top_k <= 16,
 * n_experts <= 1024, n_tokens and hidden below 2^24. */
size_t moe_tokens_workspace(int n_tokens, int top_k, int n_experts);
int moe_tokens_dispatch(const void *x, int64_t ld_x, int dtype, int n_tokens, int hidden, const int32_t *ids,
                        int top_k, int n_experts, void *rows, int64_t ld_rows, int32_t *offsets, int32_t *pos,
                        int32_t *src, int32_t *expert, void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of x: d_x[t] = sum over j of d_rows[pos[t, j]], picks in order; a token without a pick gets
 * zeros.  pos as written by moe_tokens_dispatch; n_rows: rows of d_rows (a pos outside is no pick). */
int moe_tokens_dispatch_backward(const void *d_rows, int64_t ld_rows, int64_t n_rows, int dtype, int n_tokens,
                                 int hidden, const int32_t *pos, int top_k, void *d_x, int64_t ld_x, void *stream);

/* Rows back to their tokens: out[t] = base[t] + sum over j of gate[t, j] * rows[pos[t, j]], picks in
 * order.  gate [n_tokens x top_k]; the gate of no pick is not read.  base may be NULL (zeros). */
int moe_tokens_combine(const void *rows, int64_t ld_rows, int64_t n_rows, int dtype, int n_tokens, int hidden,
                       const int32_t *pos, const float *gate, int top_k, const void *base, int64_t ld_base, void *out,
                       int64_t ld_out, void *stream);

/* Its gradients: d_rows[pos[t, j]] = gate[t, j] * d_out[t], d_gate[t, j] = <d_out[t], rows[pos[t, j]]>
 * (0 for no pick); rows of d_rows that no pick names are left as they were.  base's gradient is d_out.
 * No two picks may name one row (moe_tokens_dispatch never does that). */
int moe_tokens_combine_backward(const void *d_out, int64_t ld_d_out, const void *rows, int64_t ld_rows,
                                int64_t n_rows, int dtype, int n_tokens, int hidden, const int32_t *pos,
                                const float *gate, int top_k, void *d_rows, int64_t ld_d_rows, float *d_gate,
                                void *stream);

/* Low-rank adapters: out[i] = base[i] + scale[e] * B_e (A_e x[i]) with e = adapter[i]; where
 * adapter[i] is outside 0 .. n_adapters-1 row i has no adapter and out[i] = base[i].
 *   x [n_rows x inner], out and base [n_rows x outer] of dtype; base may be NULL (zeros);
 *   a [n_adapters x rank x inner], b [n_adapters x outer x rank] of wtype, contiguous; smaller ranks
 *   are padded with zeros;  scale [n_adapters].
 * Types: wtype = dtype, or dtype MOE_T_F32 with any wtype (the layer's own activations are fp32).
 * No row's values enter another row's result.  Rows of one adapter next to each other (a
 * request's prompt; rows in the order of moe_tokens_dispatch) share its matrices' reads; other orders
 * are as right, only slower.  workspace: moe_adapters_forward_workspace bytes (NULL if that is 0, as it
 * is for few rows), 16-byte aligned.  Where x, base or out have rows that do not start at multiples of 16
 * bytes, moe_adapters_forward_workspace_strided bytes let the call copy them to such rows first, which is
 * faster than the way it takes with less.  Many rows want a and b to start at multiples of 16 bytes too
 * (a where inner is a multiple of 8, b where rank is); otherwise either workspace gives the slower way.
 * Limits: rank <= 256; n_rows, inner and outer below 2^24. */
size_t moe_adapters_forward_workspace(int n_rows, int inner, int outer, int n_adapters, int rank);
size_t moe_adapters_forward_workspace_strided(int n_rows, int inner, int outer, int n_adapters, int rank);
int moe_adapters_forward(const void *x, int64_t ld_x, const void *base, int64_t ld_base, int dtype, int n_rows,
                         int inner, int outer, const int32_t *adapter, const void *a, const void *b, int wtype,
                         const float *scale, int n_adapters, int rank, void *out, int64_t ld_out, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Its gradients.  With v = A_e x[i], u = scale[e] * B_e^T d_out[i]:
 *   d_x[i] = dx_base[i] + A_e^T u        (dx_base, the projection's own d_x, may be NULL: zeros)
 *   d_a[e] = sum over e's rows of u x[i]^T, d_b[e] = scale[e] * sum of d_out[i] v^T
 * d_a [n_adapters x rank x inner] and d_b [n_adapters x outer x rank] are fp32 and overwritten
 * (zeros for an adapter without rows).  base's gradient is d_out; scale has none.  workspace:
 * moe_adapters_workspace bytes, 16-byte aligned; _strided as above (its way with less is many times
 * slower).  Limits: those above, n_adapters <= 1024. */
size_t moe_adapters_workspace(int n_rows, int inner, int outer, int n_adapters, int rank);
size_t moe_adapters_workspace_strided(int n_rows, int inner, int outer, int n_adapters, int rank);
int moe_adapters_backward(const void *d_out, int64_t ld_d_out, const void *x, int64_t ld_x, const void *dx_base,
                          int64_t ld_dx_base, int dtype, int n_rows, int inner, int outer, const int32_t *adapter,
                          const void *a, const void *b, int wtype, const float *scale, int n_adapters, int rank,
                          void *d_x, int64_t ld_d_x, float *d_a, float *d_b, void *workspace, size_t workspace_bytes,
                          void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TOKENS_H */
