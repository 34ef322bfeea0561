/*
 * gemm_ops — the operators of a transformer block around the product, for
 * GB300 (sm_103a), C ABI. Same library as gemm_f16.h; its conventions hold
 * here too: DEVICE pointers owned by the caller, strides in ELEMENTS, work
 * enqueued on `stream`, arguments validated before the GPU is touched, launch
 * errors returned, a bounded wait that ran out reported by
 * gemm_f16_sync_status(), kernels launched with programmatic stream
 * serialization allowed, no device memory allocated by a call.
 *
 *   gemm_linear             C = act(s_a[i] s_b[j] (A @ B)[i,j] + bias[j]) + R
 *   gemm_linear_backward    its gradients
 *   gemm_rms_norm           h = x + r, y = w h / sqrt(mean(h^2) + eps),
 *                           in 16 or 32 bits, or in 8 with a scale per row
 *   gemm_rms_norm_backward  its gradients
 *   gemm_layer_norm         h = x + r, y = w (h - mean) / sqrt(var + eps) + b,
 *                           in 16 or 32 bits, or in 8 with a scale per row
 *   gemm_layer_norm_backward  its gradients
 *   gemm_quantize_rows      rows in 8 bits with a scale each
 *   gemm_saved_backward     gemm_linear_backward from values kept in 8 bits
 *
 * An 8-bit y and its scales are an A and scale_a of gemm_linear, and an A and
 * scale_a (or pre and scale_pre) of gemm_saved_backward.
 */
#ifndef GEMM_OPS_H
#define GEMM_OPS_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (the first three are GEMM_OUT_*). */
#define GEMM_TYPE_F32 GEMM_OUT_F32
#define GEMM_TYPE_F16 GEMM_OUT_F16
#define GEMM_TYPE_BF16 GEMM_OUT_BF16
#define GEMM_TYPE_E4M3 3 /* 8-bit float: 4 exponent, 3 mantissa bits, +-448, no infinity */
#define GEMM_TYPE_I8 4   /* whole number of 8 bits, -128 .. 127 */

/* Activations. x is the value in fp32 after scales and bias.
 * RELU: x < 0 ? 0 : x (a NaN stays). GELU: x Phi(x), Phi the normal
 * distribution's cumulative function. GELU_TANH: x / (1 + exp(-2u)),
 * u = sqrt(2/pi) (x + 0.044715 x^3), the tanh form of GELU.
 * SILU: x / (1 + exp(-x)). */
#define GEMM_ACT_NONE 0
#define GEMM_ACT_RELU 1
#define GEMM_ACT_GELU 2
#define GEMM_ACT_GELU_TANH 3
#define GEMM_ACT_SILU 4

/* A matrix: element (i, j) is at data + (i*stride_row + j*stride_col) elements.
 * data == NULL: the matrix is absent, where a call allows that. */
typedef struct {
    void *data;
    int64_t stride_row, stride_col;
    int32_t type; /* GEMM_TYPE_* */
} gemm_matrix_t;

/* What follows the product in gemm_linear; absent parts are NULL / NONE. */
typedef struct {
    const void *bias;      /* [N], fp32 or C's type */
    int32_t bias_type;     /* GEMM_TYPE_*, read when bias != NULL */
    int32_t activation;    /* GEMM_ACT_* */
    const float *scale_a;  /* [M] fp32: factor of each row of A, or NULL (1) */
    const float *scale_b;  /* [N] fp32: factor of each column of B, or NULL (1) */
    gemm_matrix_t residual; /* [M, N], C's type; added after the activation */
    gemm_matrix_t pre;      /* [M, N], C's type; written: the value before the activation */
} gemm_epilogue_t;

/* flags of gemm_linear and gemm_linear_backward: 0 lets the library choose the
 * kernel by the sizes (the rule is in gemm_linear's comment below). */
#define GEMM_LINEAR_PAIR 0x1u  /* CTA pairs on 256x256 tiles */
#define GEMM_LINEAR_SPLIT 0x2u /* one CTA per 128 columns of C and 16..256 rows, K split over a cluster */
#define GEMM_LINEAR_ALL_FLAGS 0x3u

/*
 * gemm_linear — a product with its epilogue:
 *
 *   x[i,j] = scale_a[i] scale_b[j] sum_k A[i,k] B[k,j] + bias[j]
 *   pre[i,j] = x[i,j]                        (when asked for)
 *   C[i,j] = act(x[i,j]) + residual[i,j]
 *
 * The sum and everything after it are in fp32; pre and C are each rounded once
 * (nearest-even). A [M,K] and B [K,N] have one type, fp16, bf16, e4m3 or int8; C is
 * fp32, fp16 or bf16. Scales are for 8-bit operands only (both or neither). The
 * products of int8 operands are exact, and so is their sum while the sum of their
 * magnitudes stays below 2^24 (K up to 1024 whatever the values). Beyond, it is a sum
 * in fp32 on the tensor cores, not a 32-bit integer one: each addition may lose
 * 2^-23 of the magnitudes added up so far (twice what rounding to nearest loses), in
 * all (K + 16) 2^-23 sum_k |A[i,k] B[k,j]| at most, also where the sum is small.
 * Layouts: A with a unit row or column stride, B likewise (a B with stride_row
 * == 1 is a weight stored [N,K]); 8-bit operands with K contiguous only; C, pre
 * and residual with stride_col == 1 and stride_row >= N (M > 1). Others ->
 * GEMM_ERR_UNSUPPORTED / INVALID_ARG as in gemm_f16. C may be residual itself
 * (same data and strides); otherwise outputs overlap no input and no other
 * output (undefined).
 * workspace: 128-byte aligned, of gemm_linear_workspace_size() bytes, needed
 * only where that is not 0: an operand whose base or row stride is no multiple
 * of 16 bytes is first copied there onto 128-byte lines (one kernel), and int8
 * operands as fp16 (A of more than 64 rows; B too where the product's own kernel
 * takes 16 bits). Its contents mean nothing between calls.
 * M, N or K < 0 or >= 2^31 -> INVALID_ARG. M == 0 or N == 0: nothing is done.
 * K == 0: the sum is 0 and the epilogue still runs.
 * Two kernels share the work by a rule on M, N and K: 256x256 tiles on CTA
 * pairs where they keep the GPU's pairs busy; below that (few tokens: decoding,
 * short prompts; few output tiles) tiles of 128 columns by 16..256 rows with K
 * split over a cluster of up to 8 CTAs, whose partial sums are added in rank
 * order through distributed shared memory. int8 operands of up to 768 rows, and
 * small products of them, have a kernel of their own, whatever the flags.
 * Every result is deterministic.
 * The second kernel may ask for lines of B in L2 before the kernels before it on
 * the stream have ended; it uses no data of theirs before they have.
 */
gemm_status_t gemm_linear(const gemm_matrix_t *A, const gemm_matrix_t *B, const gemm_matrix_t *C,
                          const gemm_epilogue_t *epilogue, int64_t M, int64_t N, int64_t K, uint32_t flags,
                          void *workspace, uint64_t workspace_bytes, gemm_stream_t stream);

/* Workspace bytes of gemm_linear for these operands (data, strides and type are
 * looked at, nothing is read). Needs no device. */
gemm_status_t gemm_linear_workspace_size(const gemm_matrix_t *A, const gemm_matrix_t *B, int64_t M, int64_t N,
                                         int64_t K, uint64_t *bytes);

/*
 * gemm_linear_backward — gradients of gemm_linear without scales, from the
 * gradient G of C [M,N]:
 *
 *   D = G act'(pre)          (D = G without activation; act' in fp32)
 *   dA = D B^T  [M,K]        dB = A^T D  [K,N]        dbias[j] = sum_i D[i,j]
 *
 * The residual's gradient is G itself. G, pre, A and B have one 16-bit type;
 * dA and dB are fp16, bf16 or fp32, with a unit column stride or (a weight kept
 * as its transpose) a unit row stride; dbias is fp32 [N]. Each of dA, dB
 * and dbias may be absent (data == NULL). D is rounded to G's type for the two
 * products, which run on 16-bit tensor cores with fp32 sums, and not for
 * dbias. relu'(x) is 1 for x > 0, else 0. G and pre have stride_col == 1.
 * workspace: 128-byte aligned, gemm_linear_backward_workspace_size() bytes; it
 * holds D, copies of unaligned operands and partial column sums. Sizes and
 * layouts as gemm_linear. M == 0 or K == 0, N == 0: the gradients that exist
 * are zero-filled. The call's kernels may run at the same time where one needs
 * nothing of the other; what follows on the stream finds all of them complete.
 */
gemm_status_t gemm_linear_backward(const gemm_matrix_t *G, const gemm_matrix_t *A, const gemm_matrix_t *B,
                                   const gemm_matrix_t *pre, int32_t activation, const gemm_matrix_t *dA,
                                   const gemm_matrix_t *dB, float *dbias, int64_t M, int64_t N, int64_t K,
                                   uint32_t flags, void *workspace, uint64_t workspace_bytes,
                                   gemm_stream_t stream);

gemm_status_t gemm_linear_backward_workspace_size(const gemm_matrix_t *G, const gemm_matrix_t *A,
                                                  const gemm_matrix_t *B, int32_t activation, int32_t need_dbias,
                                                  int64_t M, int64_t N, int64_t K, uint64_t *bytes);

/*
 * gemm_rms_norm — for each row i of `rows`:
 *
 *   h = x[i,:] + residual[i,:]      (residual absent: h = x)
 *   rstd[i] = 1 / sqrt(mean(h^2) + eps)
 *   y[i,:] = weight * h * rstd[i]
 *
 * everything in fp32 from the unrounded sum h; h, y and rstd are each rounded
 * once. x, residual and h have one type, fp32, fp16 or bf16; y has that type or
 * e4m3; weight [width] has x's type or is fp32. With an e4m3 y, a = max_j
 * |y[i,j]|, scale[i] = a / 448 and y[i,j] holds nearest-even(y[i,j] * (448 /
 * a)), so that the value is y * scale; a row of zeros (also with eps = 0) and a
 * row whose a is below 7.7e-34 have scale 1 and zeros; a row with a NaN or an
 * infinity has scale NaN and NaNs. weight * h is a value in fp32 of its own: what
 * of it falls below fp32's smallest numbers counts as 0. scale must be given
 * with an e4m3 y, and only then.
 * h (given only with residual) may be x or residual itself. rstd may be NULL.
 * All matrices have stride_col == 1 and stride_row >= width (rows > 1).
 * rows == 0: nothing is done. width == 0: scale 1 and rstd 1 / sqrt(eps), where
 * given, are all that is written. eps >= 0, finite.
 */
gemm_status_t gemm_rms_norm(const gemm_matrix_t *x, const gemm_matrix_t *residual, const void *weight,
                            int32_t weight_type, const gemm_matrix_t *y, const gemm_matrix_t *h, float *scale,
                            float *rstd, int64_t rows, int64_t width, float eps, gemm_stream_t stream);

/*
 * gemm_rms_norm_backward — gradients of gemm_rms_norm (16- or 32-bit y) from
 * the gradient `grad` of y, h and rstd as the forward call left them, and the
 * gradient grad_h that arrives at h itself (the residual path; may be absent):
 *
 *   u = h rstd, g = grad * weight
 *   dx = rstd (g - u mean(g u)) + grad_h      (x's and residual's gradient)
 *   dweight[j] = sum_i grad[i,j] u[i,j]       (fp32 [width]; may be NULL)
 *
 * in fp32; dx is rounded once. grad, h, grad_h and dx have one type, fp32, fp16
 * or bf16. dx may be grad or grad_h itself. Sums over rows are in a fixed
 * order. workspace: 16-byte aligned, gemm_rms_norm_backward_workspace_size()
 * bytes (partial sums of dweight; needed when dweight is asked for).
 * rows == 0: dweight is zero-filled.
 */
gemm_status_t gemm_rms_norm_backward(const gemm_matrix_t *grad, const gemm_matrix_t *h, const void *weight,
                                     int32_t weight_type, const float *rstd, const gemm_matrix_t *grad_h,
                                     const gemm_matrix_t *dx, float *dweight, int64_t rows, int64_t width,
                                     void *workspace, uint64_t workspace_bytes, gemm_stream_t stream);

gemm_status_t gemm_rms_norm_backward_workspace_size(int64_t rows, int64_t width, uint64_t *bytes);

/*
 * gemm_layer_norm — for each row i of `rows`:
 *
 *   h = x[i,:] + residual[i,:]      (residual absent: h = x)
 *   mean[i] = sum(h) / width,  rstd[i] = 1 / sqrt(sum((h - mean)^2) / width + eps)
 *   y[i,:] = weight * (h - mean[i]) * rstd[i] + bias
 *
 * everything in fp32 from the unrounded sum h, the variance from the centred values,
 * whose own sum corrects a mean that is large beside it; h, y, mean and rstd are each
 * rounded once. The squares are numbers of fp32: deviations from 1e-18 to 1e18. x,
 * residual and h have one type, fp32, fp16 or bf16; y has that type or is e4m3 or int8; weight and bias
 * [width] both have x's type or both are fp32; bias may be NULL. With an 8-bit y,
 * a = max_j |y[i,j]|, scale[i] = a / t and y[i,j] holds nearest-even(y[i,j] *
 * (t / a)), t = 448 (e4m3) or 127 (int8), so that the value is y * scale; a row whose
 * a is below 7.7e-34 has scale 1 and zeros; a row with a NaN or an infinity has
 * scale NaN (and NaNs in e4m3, zeros in int8). scale must be given with an 8-bit y,
 * and only then. A row of equal values has that value as its mean and is the bias;
 * with eps = 0 it is NaN.
 * h (given only with residual) may be x or residual itself. mean and rstd may be
 * NULL. All matrices have stride_col == 1 and stride_row >= width (rows > 1).
 * rows == 0: nothing is done. width == 0: scale 1, mean 0 and rstd 1 / sqrt(eps),
 * where given, are all that is written. eps >= 0, finite.
 */
gemm_status_t gemm_layer_norm(const gemm_matrix_t *x, const gemm_matrix_t *residual, const void *weight,
                              const void *bias, int32_t weight_type, const gemm_matrix_t *y, const gemm_matrix_t *h,
                              float *scale, float *mean, float *rstd, int64_t rows, int64_t width, float eps,
                              gemm_stream_t stream);

/*
 * gemm_layer_norm_backward — gradients of gemm_layer_norm (16- or 32-bit y) from
 * the gradient `grad` of y, h, mean and rstd as the forward call left them, and the
 * gradient grad_h that arrives at h itself (the residual path; may be absent):
 *
 *   u = (h - mean) rstd, g = grad * weight
 *   dx = rstd (g - mean(g) - u mean(g u)) + grad_h   (x's and residual's gradient)
 *   dweight[j] = sum_i grad[i,j] u[i,j],  dbias[j] = sum_i grad[i,j]   (fp32 [width])
 *
 * in fp32, where rstd^2 mean(g u) has to be a number too (rstd up to 1e18); dx is
 * rounded once. grad, h, grad_h and dx have one type, fp32, fp16
 * or bf16. dx may be grad or grad_h itself. dweight and dbias may each be NULL.
 * Sums over rows are in a fixed order. workspace: 16-byte aligned,
 * gemm_layer_norm_backward_workspace_size() bytes (partial sums over the rows;
 * needed when dweight or dbias is asked for). rows == 0: both are zero-filled.
 */
gemm_status_t gemm_layer_norm_backward(const gemm_matrix_t *grad, const gemm_matrix_t *h, const void *weight,
                                       int32_t weight_type, const float *mean, const float *rstd,
                                       const gemm_matrix_t *grad_h, const gemm_matrix_t *dx, float *dweight, float *dbias,
                                       int64_t rows, int64_t width, void *workspace, uint64_t workspace_bytes,
                                       gemm_stream_t stream);

gemm_status_t gemm_layer_norm_backward_workspace_size(int64_t rows, int64_t width, uint64_t *bytes);

/*
 * gemm_quantize_rows — each row of x in 8 bits with a scale: a = max_j |x[i,j]|,
 * scale[i] = a / t, q[i,j] the value nearest to x[i,j] t / a, t = 448 (q in e4m3)
 * or 127 (int8), rows of tiny values and rows with a NaN or an infinity as in
 * gemm_layer_norm. Of two values as near the even one is taken: exactly so for x of
 * 16 bits; an fp32 x t / a is first rounded to fp32. x is fp32, fp16 or bf16, scale fp32 [rows]. q overlaps no part
 * of x. Both matrices have stride_col == 1 and stride_row >= width (rows > 1).
 * rows == 0: nothing is done. width == 0: a scale of 1 is all that is written.
 */
gemm_status_t gemm_quantize_rows(const gemm_matrix_t *x, const gemm_matrix_t *q, float *scale, int64_t rows, int64_t width,
                                 gemm_stream_t stream);

/*
 * gemm_saved_backward — gemm_linear_backward of C = act(A' @ B + bias) + R from
 * what was kept of A' [M,K] and of the values before the activation in 8 bits:
 *
 *   A'[i,k] = act_a(scale_a[i] A[i,k])     rounded to G's type
 *   D = G act'(scale_pre[i] pre[i,j])      in fp32, rounded for the products
 *   dA' = D B^T  [M,K]      dB = A'^T D  [K,N]      dbias[j] = sum_i D[i,j]
 *
 * A is e4m3 or int8 with scale_a [M] fp32 (K contiguous), or 16-bit with scale_a NULL
 * and activation_a NONE; pre likewise with scale_pre, absent with activation NONE.
 * activation_a is for a product whose operand is itself an activation: what was
 * kept is the value before it (dA' is still the gradient of act_a's result). G and B
 * are fp16 or bf16. Everything else as gemm_linear_backward, whose result this is
 * for the values that the 8 bits hold. workspace: 128-byte aligned,
 * gemm_saved_backward_workspace_size() bytes; A' is made there where dB is asked for.
 */
gemm_status_t gemm_saved_backward(const gemm_matrix_t *G, const gemm_matrix_t *A, const float *scale_a, int32_t activation_a,
                                  const gemm_matrix_t *B, const gemm_matrix_t *pre, const float *scale_pre, int32_t activation,
                                  const gemm_matrix_t *dA, const gemm_matrix_t *dB, float *dbias, int64_t M, int64_t N,
                                  int64_t K, uint32_t flags, void *workspace, uint64_t workspace_bytes,
                                  gemm_stream_t stream);

gemm_status_t gemm_saved_backward_workspace_size(const gemm_matrix_t *G, const gemm_matrix_t *A, const gemm_matrix_t *B,
                                                 int32_t activation, int32_t need_dbias, int64_t M, int64_t N, int64_t K,
                                                 uint64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_OPS_H */
