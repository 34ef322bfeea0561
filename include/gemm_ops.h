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
 *
 * An 8-bit y and its scales are an A and scale_a of gemm_linear.
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
 * (nearest-even). A [M,K] and B [K,N] have one type, fp16, bf16 or e4m3; C is
 * fp32, fp16 or bf16. Scales are for e4m3 operands only (both or neither).
 * Layouts: A with a unit row or column stride, B likewise (a B with stride_row
 * == 1 is a weight stored [N,K]); e4m3 operands with K contiguous only; C, pre
 * and residual with stride_col == 1 and stride_row >= N (M > 1). Others ->
 * GEMM_ERR_UNSUPPORTED / INVALID_ARG as in gemm_f16. C may be residual itself
 * (same data and strides); otherwise outputs overlap no input and no other
 * output (undefined).
 * workspace: 128-byte aligned, of gemm_linear_workspace_size() bytes, needed
 * only where that is not 0: an operand whose base or row stride is no multiple
 * of 16 bytes is first copied there onto 128-byte lines (one kernel). Its
 * contents mean nothing between calls.
 * M, N or K < 0 or >= 2^31 -> INVALID_ARG. M == 0 or N == 0: nothing is done.
 * K == 0: the sum is 0 and the epilogue still runs.
 * Two kernels share the work by a rule on M, N and K: 256x256 tiles on CTA
 * pairs where they keep the GPU's pairs busy; below that (few tokens: decoding,
 * short prompts; few output tiles) tiles of 128 columns by 16..256 rows with K
 * split over a cluster of up to 8 CTAs, whose partial sums are added in rank
 * order through distributed shared memory. Every result is deterministic.
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
 * rows == 0 or width == 0: nothing is done. eps >= 0, finite.
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

#ifdef __cplusplus
}
#endif

#endif /* GEMM_OPS_H */
