// Layer norm, its gradients and 8-bit rows: what the host side (ops_block.cu) hands to
// the kernels' translation unit (ops_rows.cu), which shares no device state with the
// products' one: its kernels wait for nothing but their own copies and barriers.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace g16 {

constexpr int32_t kOutSame = 0, kOutE4m3 = 1, kOutI8 = 2;  // an output's type: the input's, or 8 bits with a scale per row

// type: 0 fp32, 1 fp16, 2 bf16 (of x, r, h, grad, dx, and of weights unless w_f32).
struct LayerNormArgs {
    const void *x, *r;  // r == nullptr: no residual
    const void *w, *b;  // b == nullptr: no bias
    void *y, *h;        // h == nullptr: not stored
    float *scale, *mean, *rstd;
    int64_t rows, width;
    int64_t ldx, ldr, ldy, ldh;
    float eps, inv_width;
    int32_t w_f32, type, out;
    bool vec, shift;  // rows on 16-byte boundaries; rows that all start at the same place in a granule
};

struct LayerNormBackwardArgs {
    const void *g, *h, *dh;  // dh == nullptr: none
    const void *w;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // column sums by blocks of rows, dweight's then dbias's; nullptr: neither is asked for
    int64_t rows, width;
    int64_t ldg, ldh, lddh, lddx;
    float inv_width;
    int32_t w_f32, type;
    bool vec, shift;
};

struct QuantizeArgs {
    const void *x;
    void *q;
    float *scale;
    int64_t rows, width, ldx, ldq;
    int32_t type, out;
    bool vec, shift;
};

// Blocks whose column sums layer norm's backward pass keeps apart, at most.
constexpr int64_t kLayerNormParts = 608;

#define G16_HIDDEN __attribute__((visibility("hidden")))
G16_HIDDEN cudaError_t launch_layer_norm(const LayerNormArgs &p, int num_sms, cudaStream_t stream);
G16_HIDDEN cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs &p, float *dweight, float *dbias, int dev, int num_sms,
                                                  cudaStream_t stream);
G16_HIDDEN cudaError_t launch_quantize_rows(const QuantizeArgs &p, int num_sms, cudaStream_t stream);

#ifdef GEMM_DEBUG
// The checked build's: the source line in ops_rows.cu of the first check that failed (0: none), which is
// then forgotten; and a kernel of one failing check that guards nothing.
G16_HIDDEN cudaError_t take_rows_check_line(unsigned int *line);
G16_HIDDEN cudaError_t rows_check_selftest(cudaStream_t stream);
#endif

}  // namespace g16
