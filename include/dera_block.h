/*
 * dera_block — the rest of an encoder block around the attention of dera_relpos.h
 * and the norms and rotations of dera_train.h, in the same library:
 *   - dera_layer_norm and its backward;
 *   - dera_linear: tokens times a weight with bias, activation and residual in one
 *     kernel, and its backward;
 *   - dera_activation_backward for an activation whose input another layer made.
 * One block, in order:
 *   layer_norm, linear (packed heads), qk_norm_rope, the attention, linear (from its heads, residual),
 *   layer_norm, linear (activation), linear (residual).
 *
 * The conventions of dera_relpos.h and dera_train.h hold: device pointers of the current
 * device, 16-byte aligned unless an entry says otherwise; row-major contiguous layouts unless strides are
 * given; the caller owns every buffer; nothing allocates or synchronises; all work goes to `stream`
 * and can be captured in a graph; argument errors are found on the host before anything is
 * enqueued; a call without rows returns before any pointer is looked at (but for gradients of
 * parameters, which are then written as zeros).  Outputs may not overlap inputs or one another.  A
 * workspace is 256-byte aligned device memory that no other call in flight uses (two graphs that
 * may run at the same time each need their own); its contents need no initialisation.  Nothing is
 * accumulated with atomics: every result is the same on every run.
 */
#ifndef DERA_BLOCK_H
#define DERA_BLOCK_H

#include "dera_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm.  Per row x of `cols` values:
 *     mean = sum(x) / cols,  rstd = 1 / sqrt(sum((x - mean)^2) / cols + eps),
 *     y = (x - mean) rstd weight + bias                 (weight 1 and bias 0 where they are NULL)
 * in fp32, the variance from centred values, y rounded once.  A row's sum, and the sum of its squared deviations, have to stay
 * within fp32's range; an infinity or NaN makes its own row NaN and no other.
 * in:  x [rows, cols] in in_dtype (any of the three), its rows x_stride >= cols elements apart (not looked at for one
 *      row); weight, bias [cols] in weight_dtype (DERA_F32 or the 16-bit type of in_dtype or out_dtype).
 * out: y [rows, cols] in out_dtype (DERA_F32, in_dtype, or any type where in_dtype is DERA_F32); mean, rstd [rows] fp32.
 * Pointers need the alignment of their elements only; rows of a multiple of 8 columns at 16-byte addresses are
 * faster (all of x, y, and x_stride).
 * Errors: DERA_ERR_SHAPE for rows < 0, cols outside [1, 16384], x_stride < cols, eps negative or not finite;
 *      DERA_ERR_NULL for a bias without a weight.
 */
DERA_API dera_status dera_layer_norm(const void* x, const void* weight, const void* bias, void* y, float* mean,
                              float* rstd, int rows, int cols, long long x_stride, float eps, dera_dtype in_dtype,
                              dera_dtype weight_dtype, dera_dtype out_dtype, void* stream);

/* Scratch of dera_layer_norm_backward on the current device (partial weight gradients). */
DERA_API dera_status dera_layer_norm_backward_workspace_size(int rows, int cols, size_t* bytes);

/*
 * Backward of dera_layer_norm.  With h = (x - mean) rstd and g = dy weight, per row:
 *     dx = rstd (g - mean(g) - h mean(g h)) + dres,   dweight = sum over rows of dy h,   dbias = sum of dy.
 * in:  x, weight as given to the forward, mean and rstd as it gave them; dy [rows, cols] in dout_dtype (DERA_F32,
 *      in_dtype, or any where in_dtype is DERA_F32); dres [rows, cols] in grad_dtype, a gradient that reaches x past the
 *      norm (the residual's), or NULL.
 * out: dx [rows, cols] in grad_dtype (DERA_F32 or in_dtype); dweight, dbias [cols] fp32, both or (NULL) neither.
 * workspace: at least the size above if dweight is given (else it may be NULL).
 * Alignment and errors as for the forward; DERA_ERR_SCRATCH for a missing or too small workspace.  rows = 0 writes zero
 * dweight and dbias.
 */
DERA_API dera_status dera_layer_norm_backward(const void* dy, const void* x, const float* mean, const float* rstd,
                              const void* weight, const void* dres, void* dx, float* dweight, float* dbias, int rows,
                              int cols, long long x_stride, dera_dtype in_dtype, dera_dtype weight_dtype,
                              dera_dtype dout_dtype, dera_dtype grad_dtype, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Activations of a linear layer, act(u), all in fp32. */
typedef enum dera_activation {
  DERA_ACT_NONE = 0,
  DERA_ACT_RELU = 1,        /* max(u, 0) */
  DERA_ACT_GELU = 2,        /* u Phi(u), Phi the normal distribution */
  DERA_ACT_GELU_TANH = 3,   /* u / 2 (1 + tanh(sqrt(2 / pi) (u + 0.044715 u^3))) */
  DERA_ACT_QUICK_GELU = 4,  /* u / (1 + exp(-1.702 u)) */
  DERA_ACT_SILU = 5         /* u / (1 + exp(-u)) */
} dera_activation;

/*
 * A linear layer over B * N tokens of K = heads * head_dim features:
 *     u = x weight^T + bias,   y = act(u) + residual.
 * in:  x by its strides (elements, as in dera_train.h: >= 0 here only where the dimension has size one, else positive
 *      multiples of 8): plain rows are heads = 1, head_dim = K; the [B * heads, N, head_dim] that the
 *      attention gives are strides (heads N head_dim, head_dim, N head_dim), read as they lie.  weight
 *      [out_features, K]; both in in_dtype (DERA_F16 | DERA_BF16).  bias [out_features] in bias_dtype (DERA_F32 or
 *      in_dtype), or NULL.  residual [B, N, out_features] in out_dtype, or NULL.
 * out: y [B, N, out_features] in out_dtype (DERA_F32 or in_dtype); pre, if not NULL, u in in_dtype (what the backward of
 *      the activation needs).
 * K and out_features are multiples of 8, head_dim of 64 where heads > 1.  Sums are fp32.  The tensor core cuts towards zero
 * when it adds: 16 products a step, each at a quarter of a unit in the last place of the sum so far, and the new sum at a whole one, at
 * most 5 2^-23 of a partial sum.  In sums of one sign this adds up, to 6.4e-9 a term for fp16 and 3.6e-9 for bf16, whose products have fewer
 * bits (measured; relative to the sum of the terms' sizes); mixed signs cancel.  Where y is fp32 no more than 512 terms are added so
 * (2.8e-6 off on average for fp16 terms of one sign and 9e-7 for bf16, 3.7e-6 and 1.5e-6 at most), and these sums with rounding; where y has 16
 * bits, up to all K: below half a step of y for fp16 up to K = 75000, and for bf16.  Bias,
 * activation and residual are applied in fp32, and y (and pre) rounded once.  x and weight must be finite.  Gelu's Phi(u) is off by
 * 2^-18 + u^2 2^-23 of its distance to 0 or 1 (measured: 1.2e-6 of it up to |u| = 2, 2e-6 up to 6, 4.4e-6 up to 10, 6.5e-6 up to 13); an
 * element's last bit may depend on its neighbour's.
 * Errors: DERA_ERR_SHAPE for sizes below one (B = 0 or N = 0 is a no-op), B * N beyond 2^31 - 1, features beyond 2^20,
 *      features or strides that break the rules above; DERA_ERR_ALIGN for strides that are not multiples of 8;
 *      DERA_ERR_DTYPE also for an unknown activation.
 */
DERA_API dera_status dera_linear(const dera_heads* x, const void* weight, const void* bias, const void* residual, void* y,
                              void* pre, int B, int N, int heads, int head_dim, int out_features,
                              dera_activation activation, dera_dtype in_dtype, dera_dtype bias_dtype,
                              dera_dtype out_dtype, void* stream);

/* Scratch of dera_linear_backward on the current device. */
DERA_API dera_status dera_linear_backward_workspace_size(int B, int N, int heads, int head_dim, int out_features,
                              size_t* bytes);

/*
 * Backward of x weight^T + bias, with dy its gradient (the residual's is dy itself):
 *     dx = (dy weight) * act'(input_pre),   dweight = dy^T x,   dbias = sum over tokens of dy.
 * With input_pre the layer's input is taken as x = act(input_pre), the activation of the layer
 * before, and dx is the gradient of input_pre; without it (NULL, DERA_ACT_NONE) of x.
 * in:  dy [B, N, out_features], x and input_pre (by their strides) and weight in in_dtype.
 * out: dx with the strides given, in grad_dtype, dweight [out_features, K] in weight_grad_dtype (DERA_F32 or in_dtype each),
 *      dbias [out_features] fp32.  Any of the three may be NULL: it is not computed (x is needed for dweight,
 *      weight for dx only).
 * workspace: at least the size above if dweight or dbias is given (else it may be NULL).
 * Precision as for dera_linear.  Errors as for dera_linear, DERA_ERR_SCRATCH for a missing or too small workspace; B = 0 or
 *      N = 0 writes zero dweight and dbias.
 */
DERA_API dera_status dera_linear_backward(const void* dy, const dera_heads* x, const void* weight,
                              const dera_heads* input_pre, const dera_heads* dx, void* dweight, float* dbias, int B, int N,
                              int heads, int head_dim, int out_features, dera_activation input_activation,
                              dera_dtype in_dtype, dera_dtype grad_dtype, dera_dtype weight_grad_dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Backward of an activation: dpre[i] = dy[i] act'(pre[i]) for n elements, in fp32, rounded once.
 * in:  dy in dout_dtype (DERA_F32 or pre_dtype), pre in pre_dtype (any of the three).
 * out: dpre in grad_dtype (DERA_F32 or pre_dtype).
 * Errors: DERA_ERR_SHAPE for n < 0; DERA_ERR_DTYPE also for DERA_ACT_NONE or an unknown activation.  n = 0 is a no-op.
 */
DERA_API dera_status dera_activation_backward(const void* dy, const void* pre, void* dpre, long long n,
                              dera_activation activation, dera_dtype pre_dtype, dera_dtype dout_dtype,
                              dera_dtype grad_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DERA_BLOCK_H */
