/*
 * dera_train — what a training step (or a step of single new tokens) needs
 * around the attention of dera_relpos.h, in the same library:
 *   - dera_qk_norm_rope: the heads of the packed projection, normed, rotated and
 *     laid out as the attention takes them, and its backward;
 *   - dera_relpos_attention_lse: the compact-bias attention that also writes its
 *     log-sum-exp, and dera_relpos_attention_backward (head_dim 64 or 128);
 *   - dera_relpos_project_backward: from the compact bias's gradient to the
 *     tables' and q's.
 * One step of the two-step form, in order:
 *   qk_norm_rope, project, attention_lse | attention_backward, project_backward, qk_norm_rope_backward.
 *
 * The conventions of dera_relpos.h hold: device pointers of the current device,
 * 16-byte aligned; row-major contiguous layouts unless strides are given; the
 * caller owns every buffer; nothing allocates or synchronises; all work goes to
 * `stream` and can be captured in a graph; argument errors are found on the host
 * before anything is enqueued; an empty batch returns before any pointer is looked at
 * (but for gradients of shared parameters, which are then written as zeros).
 * Outputs may not overlap inputs or one another unless an entry says so.  A
 * workspace is 256-byte aligned device memory that no other call in flight uses
 * (two graphs that may run at the same time each need their own); its contents
 * need no initialisation.  Nothing is accumulated with atomics: every result is the
 * same on every run.
 */
#ifndef DERA_TRAIN_H
#define DERA_TRAIN_H

#include "dera_relpos.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Heads as a projection leaves them: element (b, n, h, c) of a [B, N, heads, head_dim]
 * tensor is data[b * stride_batch + n * stride_token + h * stride_head + c], strides in
 * elements, >= 0 and multiples of 8 (16-byte rows; fp32 gradients too).  The stride of a
 * dimension of size one is not looked at.  A slice of a packed [B, N, q + k + v heads,
 * head_dim] buffer is one of these.  Inputs may repeat rows (stride 0); the rows of an
 * output must not overlap.
 */
typedef struct dera_heads {
  void* data;
  long long stride_batch, stride_token, stride_head;
} dera_heads;

/*
 * Norms of queries and keys for each head and the rotation by position, in one pass
 * that also brings q, k and v from token order to the [B * heads, N, head_dim] that
 * project, attention and fused take.  Per row x of head_dim values (one token, one head):
 *     y = x / sqrt(mean(x^2) + eps) * weight          (y = x without weights)
 *     z_a = y_a cos_i - y_b sin_i,  z_b = y_b cos_i + y_a sin_i     for i < rotary_dim / 2,
 * where the pair (a, b) is (i, i + rotary_dim / 2), or (2i, 2i + 1) if `interleaved`; elements
 * from rotary_dim on pass.  cos_i, sin_i come from row p of the tables, p = positions[b, n], or
 * n without positions (so a 64x64 grid's two-axis angles are a table of 4096 rows).  v is moved
 * as it is.  Computed in fp32 and rounded once (2 mean(x^2) has to stay within fp32's range).
 * in:  q [B,N,q_heads,head_dim], k and (or NULL) v [B,N,kv_heads,head_dim] in in_dtype (DERA_F16 | DERA_BF16);
 *      q_weight, k_weight [head_dim] in weight_dtype (DERA_F32 or in_dtype), both or neither;
 *      cos, sin [table_rows, rotary_dim / 2] fp32, both iff rotary_dim > 0; positions [B,N]
 *      int32 or NULL.
 * out: q_out [B*q_heads,N,head_dim], k_out [B*kv_heads,N,head_dim], v_out (iff v) likewise, in_dtype.
 * rotary_dim: 0 or a multiple of 16 up to head_dim.  Without positions table_rows >= N.
 * A position outside [0, table_rows) reads nothing: every rotated element of that token is NaN.
 * Errors: DERA_ERR_HEAD_DIM unless head_dim is 64 or 128; DERA_ERR_SHAPE for sizes below one (B = 0 or
 *      N = 0 is a no-op), B * N beyond 2^31 - 1, more than 16384 heads, rotary_dim, table_rows or a
 *      stride that break the rules above, eps negative or not finite; DERA_ERR_ALIGN for a stride that is
 *      not a multiple of 8; DERA_ERR_NULL for one of a pair that belongs together.
 */
DERA_API dera_status dera_qk_norm_rope(const dera_heads* q, const dera_heads* k, const dera_heads* v,
                              const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                              const int* positions, void* q_out, void* k_out, void* v_out, int B, int N, int q_heads,
                              int kv_heads, int head_dim, int rotary_dim, int table_rows, int interleaved, float eps,
                              dera_dtype in_dtype, dera_dtype weight_dtype, void* stream);

/* Scratch of dera_qk_norm_rope_backward on the current device (partial weight gradients). */
DERA_API dera_status dera_qk_norm_rope_backward_workspace_size(int B, int N, int q_heads, int kv_heads, int head_dim,
                              size_t* bytes);

/*
 * Backward of dera_qk_norm_rope.  With dz the gradient of q_out (k_out), y' = R^T dz (the
 * rotation by the negative angle), r = 1 / sqrt(mean(x^2) + eps) and g = y' weight, per row:
 *     dx = r (g - x r^2 mean(g x)),   dweight = sum over rows of y' x r
 * (dx = y' without weights).  fp32 throughout, dx rounded once.
 * in:  q, k as given to the forward (NULL without weights: only the norm needs them); dq_out, dk_out and
 *      (or NULL) dv_out, laid out as q_out, k_out, v_out, in dout_dtype (DERA_F32 or in_dtype).
 * out: dq, dk and (iff dv_out) dv in token order with the strides given, in grad_dtype
 *      (DERA_F32 or in_dtype); dq_weight, dk_weight [head_dim] fp32, iff weights.
 * workspace: at least the size above if weights are given (else it may be NULL).
 * An out-of-range position gives NaN as in the forward, in that token's gradients and so in the weights'.
 * Other arguments and errors as for the forward;
 *      DERA_ERR_SCRATCH for a missing or too small workspace.  B = 0 or N = 0 writes zero weight gradients.
 */
DERA_API dera_status dera_qk_norm_rope_backward(const dera_heads* q, const dera_heads* k, const void* q_weight,
                              const void* k_weight, const float* cos, const float* sin, const int* positions,
                              const void* dq_out, const void* dk_out, const void* dv_out, const dera_heads* dq,
                              const dera_heads* dk, const dera_heads* dv, float* dq_weight, float* dk_weight, int B,
                              int N, int q_heads, int kv_heads, int head_dim, int rotary_dim, int table_rows,
                              int interleaved, float eps, dera_dtype in_dtype, dera_dtype weight_dtype,
                              dera_dtype dout_dtype, dera_dtype grad_dtype, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * Training forward of the two-step form: dera_relpos_attention that also writes every row's base-2
 * log-sum-exp, lse[b, n] = log2(sum_m exp(Z[b, n, m])), Z = scale q k^T + rel_h + rel_w, [BH, N] fp32.
 * A bias of -inf masks its keys, and so does one of -1e38 (rounded to its type) or below, here, in
 * dera_relpos_attention and in the backward; a row with every key masked gives out = 0 and lse = -inf.  q, k and v
 * must be finite everywhere, at masked keys too (the products read them), and a bias at most 8e37 and not NaN.
 * Everything else as for dera_relpos_attention (workspace: dera_relpos_workspace_size).
 */
DERA_API dera_status dera_relpos_attention_lse(const void* q, const void* k, const void* v, const void* rel_h,
                              const void* rel_w, void* out, float* lse, int BH, int H, int W, int head_dim,
                              float scale, dera_dtype in_dtype, dera_dtype bias_dtype, dera_dtype out_dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Scratch of dera_relpos_attention_backward for a problem size on the current device. */
DERA_API dera_status dera_relpos_attention_backward_workspace_size(int BH, int H, int W, int head_dim, size_t* bytes);

/*
 * Backward of dera_relpos_attention.  With Z as above, P = softmax(Z) recomputed from lse
 * (P = 0 in a row whose lse is -inf), D[n] = dout[n] . out[n] and dZ = P * (dout v^T - D):
 *   dv = P^T dout,  dk = scale dZ^T q,  dq = scale dZ k,
 *   drel_h[n, kh] = sum_kw dZ[n, kh W + kw],  drel_w[n, kw] = sum_kh dZ[n, kh W + kw].
 * lse is fp32, so that P is off by up to 2^-24 |lse| (times ln 2, relative): nothing for logits of ordinary size, 6e-4 in
 * a row whose every key has a bias of -1e4.  A row whose lse is -2^20 or below (-1e9 on every key, say) counts as
 * masked as a whole, P = 0: rows without keys are best given as -inf.
 * in:  q, k, v, rel_h, rel_w as given to the forward, out [BH,N,head_dim] and lse [BH,N] as it gave
 *      them (out in out_dtype: DERA_F32 or in_dtype), dout [BH,N,head_dim] in in_dtype, finite everywhere.
 * out: dq, dk, dv [BH,N,head_dim] in grad_dtype (DERA_F32 or in_dtype); drel_h [BH,N,H],
 *      drel_w [BH,N,W] fp32.
 * Precision: P, dZ and the sums are fp32; P and dZ are rounded to in_dtype (relative 2^-8 for
 *      bf16, 2^-11 for fp16) as operands of the products dv, dk and dq, whose accumulators are
 *      fp32; drel_h and drel_w are summed before that rounding.  With fp16 a P or dZ below 2^-25 is
 *      lost there and a |dZ| of 65520 or more overflows.  On a grid of one row (column) drel_h (drel_w) is 0
 *      by mathematics (the softmax does not see a term that all keys share), and written as exact zeros.
 * Errors: as for dera_relpos_attention; DERA_ERR_SCRATCH if the workspace is NULL or smaller
 *      than the size above; DERA_ERR_SHAPE if BH * ceil(N / 128) passes 2^30.
 */
DERA_API dera_status dera_relpos_attention_backward(const void* q, const void* k, const void* v, const void* rel_h,
                              const void* rel_w, const void* out, const float* lse, const void* dout, void* dq,
                              void* dk, void* dv, float* drel_h, float* drel_w, int BH, int H, int W, int head_dim,
                              float scale, dera_dtype in_dtype, dera_dtype bias_dtype, dera_dtype out_dtype,
                              dera_dtype grad_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Scratch of dera_relpos_project_backward on the current device (partial table gradients). */
DERA_API dera_status dera_relpos_project_backward_workspace_size(int BH, int H, int W, int head_dim, size_t* bytes);

/*
 * Backward of dera_relpos_project.  With the gradient of the compact bias, drel_h [BH,N,H] and
 * drel_w [BH,N,W] in fp32:
 *   dq[b, n] = dq_in[b, n] + sum_kh drel_h[b, n, kh] rel_pos_h[qh - kh + H - 1]
 *                          + sum_kw drel_w[b, n, kw] rel_pos_w[qw - kw + W - 1],
 *   drel_pos_h[i] = sum over (b, n, kh) with qh - kh + H - 1 = i of drel_h[b, n, kh] q[b, n]  (same for w).
 * in:  q [BH,N,head_dim] and the tables in in_dtype; dq_in [BH,N,head_dim] in grad_dtype (the
 *      attention's own part of dq), or NULL for none; it may be dq itself.
 * out: dq [BH,N,head_dim] in grad_dtype (DERA_F32 or in_dtype); drel_pos_h [2H-1,head_dim], drel_pos_w
 *      [2W-1,head_dim] fp32, summed over every batch and head.
 * q, the tables, drel_h and drel_w must be finite everywhere (a table row's sum reads every token's q).
 * Precision: fp32 sums; drel_h and drel_w enter the products as three bf16 terms each (what is left
 *      out is 2^-24 of a value), two (2^-16) for a 16-bit dq, and with fp16 q and the tables as two
 *      bf16 terms, exactly.
 * Errors: as for dera_relpos_project; DERA_ERR_SCRATCH as above.  BH = 0 writes zero table gradients.
 */
DERA_API dera_status dera_relpos_project_backward(const void* q, const void* rel_pos_h, const void* rel_pos_w,
                              const float* drel_h, const float* drel_w, const void* dq_in, void* dq, float* drel_pos_h,
                              float* drel_pos_w, int BH, int H, int W, int head_dim, dera_dtype in_dtype,
                              dera_dtype grad_dtype, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DERA_TRAIN_H */
