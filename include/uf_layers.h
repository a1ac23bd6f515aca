/*
 * uf_layers.h -- C ABI of the operators around the contrastive loss: the trainable head that
 * makes the embeddings (RMS norm with the residual's addition, linear projections, the gated
 * feed-forward block), forward and backward, and the AdamW step that follows the gradients.
 *
 * Conventions are those of uf_contrastive.h: the caller owns every buffer and the scratch,
 * a call only enqueues kernels on the caller's stream (it can be captured in a CUDA graph) and
 * returns a uf_status_t, argument errors are found on the host before anything is enqueued, and
 * no buffer that a call writes may overlap another such buffer or an input (uf_adamw_step
 * updates its buffers in place).  The extent of a strided matrix is rows x ld without the last
 * row's tail.  All matrices are row-major; ld arguments are in elements.  Operands are bf16 or
 * e4m3, every product, sum and statistic fp32.
 *
 * Matrix products (uf_linear_*, uf_gated_*) need 16-byte aligned rows: their pointers and the
 * byte strides of their matrices are multiples of 16, and their widths (inner, outer) multiples
 * of 8, or of 16 for e4m3; bias and w_scale are 16-byte aligned.  The number of rows is free,
 * and 0 rows are a valid request that writes what an empty sum is (zero weight gradients).
 */
#ifndef UF_LAYERS_H_
#define UF_LAYERS_H_

#include "uf_contrastive.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum uf_dtype { UF_BF16 = 0, UF_F32 = 1, UF_E4M3 = 2 } uf_dtype_t;

typedef enum uf_activation {
  UF_ACT_NONE = 0,
  UF_ACT_RELU = 1,
  UF_ACT_GELU = 2,      /* z Phi(z), by erf */
  UF_ACT_GELU_TANH = 3, /* its tanh form: z sigmoid(sqrt(8/pi) (z + 0.044715 z^3)) */
  UF_ACT_SILU = 4       /* z sigmoid(z) */
} uf_activation_t;

/*
 * RMS norm with the residual's addition.  For every row, in fp32:
 *   s = x + residual;  rho = 1 / sqrt(mean(s^2) + eps);  y = s rho weight.
 *   x            [rows][width], x_type UF_BF16, or (without a residual) UF_F32.
 *   residual     [rows][width] of stream_type (UF_BF16 or UF_F32), or NULL.
 *   weight       [width], weight_type UF_BF16 or UF_F32.
 *   y            [rows][width], y_type UF_BF16, or UF_E4M3: then y = e4m3(448 y / a) with
 *                a = max |y| over the row, and y_scale[row] = a / 448 (a row of zeros, or with
 *                a < 2^-116: 0, codes 0).
 *   stream_out   [rows][width] of stream_type: s (needed with a residual, NULL without).
 *   rstd         [rows] or NULL: rho, for the backward.
 * 1 <= width <= 16384, any width and alignment of the elements' own size; rows of 16 bytes'
 * alignment take wide loads.
 */
UF_API uf_status_t uf_rmsnorm_fwd(const void* x, int64_t ldx, int x_type, const void* residual, int64_t ldr,
                                  int stream_type, const void* weight, int weight_type, int64_t rows, int width,
                                  float eps, void* y, int64_t ldy, int y_type, float* y_scale, void* stream_out,
                                  int64_t lds, float* rstd, void* stream);

/*
 * Its backward in s and the weight (dx is the gradient of both x and the residual):
 *   g = dy weight, xh = s rstd:  dx = rstd (g - xh mean(g xh)) + d_stream;  dweight = sum_rows dy xh.
 *   dy           [rows][width], dy_type UF_BF16 or UF_F32.
 *   s            [rows][width] of stream_type, the forward's stream_out (or its x, without a residual).
 *   d_stream     [rows][width] of stream_type or NULL: the gradient that reaches s past the norm.
 *   dx           [rows][width] of stream_type.
 *   dweight      [width] fp32, or NULL.
 *   workspace    uf_rmsnorm_bwd_workspace(rows, width) bytes, 256-byte aligned (may be NULL without dweight).
 */
UF_API size_t uf_rmsnorm_bwd_workspace(int64_t rows, int width);
UF_API uf_status_t uf_rmsnorm_bwd(const void* dy, int64_t lddy, int dy_type, const void* s, int64_t lds,
                                  int stream_type, const void* weight, int weight_type, const float* rstd,
                                  const void* d_stream, int64_t ldds, int64_t rows, int width, void* dx, int64_t lddx,
                                  float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Linear projection with its epilogue:  z = x W^T (+ bias);  y = act(z) (+ residual).
 *   x            [rows][inner], W [outer][inner], both of type UF_BF16 or UF_E4M3.
 *   x_scale      UF_E4M3: [rows] fp32, and w_scale [outer] fp32: element (i, j) of the product is
 *                multiplied by x_scale[i] w_scale[j] (NULL for UF_BF16).
 *   bias         [outer], bias_type UF_BF16 or UF_F32, or NULL.
 *   residual     [rows][outer] bf16 or NULL.
 *   y            [rows][outer] bf16.
 *   pre          [rows][outer] bf16 or NULL: z, for the backward.
 *   workspace    uf_linear_fwd_workspace(rows, inner, outer, type) bytes, 256-byte aligned (0: NULL is fine).
 *   device_status as in uf_contrastive_fwd_bwd.
 */
UF_API size_t uf_linear_fwd_workspace(int64_t rows, int inner, int outer, int type);
UF_API uf_status_t uf_linear_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int type,
                                 const float* x_scale, const float* w_scale, const void* bias, int bias_type,
                                 const void* residual, int64_t ldr, int act, int64_t rows, int inner, int outer,
                                 void* y, int64_t ldy, void* pre, int64_t ldp, void* workspace,
                                 size_t workspace_bytes, int* device_status, void* stream);

/*
 * Its backward (bf16 operands):  dz = dy act'(z);  dx = dz W;  dW = dz^T x;  dbias = sum_rows dz.
 * (The residual's gradient is dy itself.)  dz is rounded to bf16 for the products; dbias sums it
 * unrounded.
 *   dy           [rows][outer], dy_type UF_BF16 or UF_F32.
 *   pre          [rows][outer] bf16: the forward's z; needed unless act is UF_ACT_NONE.
 *   dx           [rows][inner] bf16, dW [outer][inner] bf16, dbias [outer] fp32: each may be NULL.
 *   workspace    uf_linear_bwd_workspace(rows, inner, outer) bytes, 256-byte aligned.
 */
UF_API size_t uf_linear_bwd_workspace(int64_t rows, int inner, int outer);
UF_API uf_status_t uf_linear_bwd(const void* dy, int64_t lddy, int dy_type, const void* x, int64_t ldx, const void* W,
                                 int64_t ldw, const void* pre, int64_t ldp, int act, int64_t rows, int inner, int outer,
                                 void* dx, int64_t lddx, void* dW, int64_t lddw, float* dbias, void* workspace,
                                 size_t workspace_bytes, int* device_status, void* stream);

/*
 * Gated feed-forward block: both projections, the activation and their product in one kernel.
 *   [g | u] = x W^T;  h = act(g) u.
 *   x            [rows][inner] bf16;  W [2 outer][inner] bf16: the gate's rows, then the up projection's.
 *   act          any but UF_ACT_NONE.
 *   h            [rows][outer] bf16.
 *   pre          [rows][2 outer] bf16 or NULL: [g | u], for the backward.
 */
UF_API size_t uf_gated_fwd_workspace(int64_t rows, int inner, int outer);
UF_API uf_status_t uf_gated_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int act, int64_t rows, int inner,
                                int outer, void* h, int64_t ldh, void* pre, int64_t ldp, void* workspace,
                                size_t workspace_bytes, int* device_status, void* stream);

/*
 * Its backward:  dg = dh u act'(g), du = dh act(g) (rounded to bf16);  dx = [dg | du] W;
 * dW = [dg | du]^T x.
 *   dh           [rows][outer] bf16;  pre [rows][2 outer] bf16.
 *   dx           [rows][inner] bf16, dW [2 outer][inner] bf16: each may be NULL.
 */
UF_API size_t uf_gated_bwd_workspace(int64_t rows, int inner, int outer);
UF_API uf_status_t uf_gated_bwd(const void* dh, int64_t lddh, const void* x, int64_t ldx, const void* W, int64_t ldw,
                                const void* pre, int64_t ldp, int act, int64_t rows, int inner, int outer, void* dx,
                                int64_t lddx, void* dW, int64_t lddw, void* workspace, size_t workspace_bytes,
                                int* device_status, void* stream);

/*
 * One AdamW step over n tensors (decoupled weight decay), in place.  With g = grad * grad_scale:
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2;
 *   p -= lr (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay p).
 * Host arrays of n device pointers each; they are read before the call returns.  What is written
 * (all but the gradients) may not overlap across tensors either: a parameter listed twice is refused.
 * Tensors may share a gradient.
 *   p            parameters, param_type UF_F32 or UF_BF16 (bf16: rounded stochastically).
 *   g            gradients, grad_type UF_F32 or UF_BF16.
 *   m, v         state_type UF_F32: fp32.  UF_E4M3: codes of m and of sqrt(v), with fp32 scales
 *                m_scale, v_scale [ceil(size / 256)] for blocks of 256 elements (value = code x
 *                scale; the block's largest magnitude is code 448), rounded stochastically so that
 *                m and v are unbiased: one step moves v by less than half a code, which
 *                rounding to nearest would drop.
 *   copy         UF_F32 parameters: bf16 copies of the new parameters, or NULL (or NULL entries).
 *   sizes        elements of each tensor (0 is allowed).
 *   beta1, beta2 doubles, so that 1 - beta is not the difference of two rounded numbers.
 *   lr, lr_dev   learning rate; lr_dev: device fp32 scalar read by the kernel instead, or NULL.
 *   step, step_dev  t >= 1; step_dev: device int64 scalar read by the kernel instead, or NULL.  With
 *                step_dev a captured CUDA graph follows the count.
 *   seed         of the stochastic rounding (with step_dev the count is added to it): give every
 *                step its own.  Element i of tensor k draws h = H(i + H(seed + 0x9E3779B9 k)), all
 *                mod 2^32, H the two-multiplication integer hash (x ^= x >> 16; x *= 0x7feb352d;
 *                x ^= x >> 15; x *= 0x846ca68b; x ^= x >> 16; from C. Wellons, Prospecting for Hash
 *                Functions, 2018); m takes its low 16 bits, v its high
 *                ones, a bf16 parameter the low 16 of H(h ^ 0x9E3779B9).
 *   grad_scale_dev  device fp32 scalar (a clipping or unscaling factor), or NULL for 1.
 */
UF_API uf_status_t uf_adamw_step(int n, void* const* p, const void* const* g, void* const* m, void* const* v,
                                 float* const* m_scale, float* const* v_scale, void* const* copy, const int64_t* sizes,
                                 int param_type, int grad_type, int state_type, float lr, const float* lr_dev,
                                 double beta1, double beta2, float eps, float weight_decay, int64_t step,
                                 const int64_t* step_dev, uint32_t seed, const float* grad_scale_dev, void* stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* UF_LAYERS_H_ */
