// Host side of layer norm and of rows in 8 bits (declared in include/gemm_ops.h):
// argument validation; the kernels and their launch shapes are in ops_rows.cu, a
// translation unit of their own. Compiled in one translation unit with ops.cu (library.cu).
#include "ops_rows.h"

namespace {

// Which of the row kernels' two vector forms the arrays of a call allow.
struct Places {
    bool vec = true, shift = true;
    const void *first;
    int64_t ld, rows;
    Places(const void *data, int64_t ld_, int es, int64_t rows_, int64_t width, std::initializer_list<const void *> columns,
           bool columns_f32)
        : first(data), ld(ld_), rows(rows_) {
        vec = width % 8 == 0 && vec16(data, ld_, es);
        shift = es == 2 && !columns_f32;
        for (const void *c : columns) {
            if (c == nullptr) continue;
            vec = vec && aligned16(c);
            shift = shift && aligned16(c);
        }
    }
    // another matrix with elements of es bytes
    void also(const void *data, int64_t ld_, int es) {
        if (data == nullptr) return;
        vec = vec && (es == 1 ? (reinterpret_cast<uintptr_t>(data) & 7u) == 0 && ld_ % 8 == 0 : vec16(data, ld_, es));
        shift = shift && same_places(first, ld, data, ld_, es, rows);
    }
};

int32_t out_code(int32_t type, int32_t x) { return type == x ? g16::kOutSame : type == GEMM_TYPE_I8 ? g16::kOutI8 : g16::kOutE4m3; }

}  // namespace

extern "C" {

gemm_status_t gemm_layer_norm(const gemm_matrix_t *x, const gemm_matrix_t *residual, const void *weight,
                              const void *bias, int32_t weight_type, const gemm_matrix_t *y, const gemm_matrix_t *h,
                              float *scale, float *mean, float *rstd, int64_t rows, int64_t width, float eps,
                              gemm_stream_t stream) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(rows, width, 0) || x == nullptr || y == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!is_c_type(x->type) || (y->type != x->type && !is_eight(y->type))) return GEMM_ERR_INVALID_ARG;
    if (weight_type != GEMM_TYPE_F32 && weight_type != x->type) return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps <= 3.0e38f)) return GEMM_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_OK;
    if (width == 0) {  // rows of no values (whose matrices may have no address): what stands beside them
        if (!words_aligned({scale, mean, rstd})) return GEMM_ERR_INVALID_ARG;
        return empty_rows(scale, mean, rstd, rows, eps, reinterpret_cast<cudaStream_t>(stream));
    }
    if (x->data == nullptr || y->data == nullptr || weight == nullptr || is_eight(y->type) != (scale != nullptr))
        return GEMM_ERR_INVALID_ARG;
    if (present(h) && !present(residual)) return GEMM_ERR_INVALID_ARG;
    if (!element_aligned(weight, weight_type) || !element_aligned(bias, weight_type) || !words_aligned({scale, mean, rstd}))
        return GEMM_ERR_INVALID_ARG;
    for (const gemm_matrix_t *m : {x, residual, y, h}) {
        if (!present(m)) continue;
        if (m != y && m->type != x->type) return GEMM_ERR_INVALID_ARG;
        const gemm_status_t st = check_rows(m, rows, width);
        if (st != GEMM_OK) return st;
    }
    DeviceState *ds = nullptr;
    if (device_state(&ds) < 0) return GEMM_ERR_CUDA;
    g16::LayerNormArgs p;
    std::memset(&p, 0, sizeof(p));
    p.x = x->data;
    p.ldx = x->stride_row;
    p.r = present(residual) ? residual->data : nullptr;
    p.ldr = present(residual) ? residual->stride_row : 0;
    p.y = y->data;
    p.ldy = y->stride_row;
    p.h = present(h) ? h->data : nullptr;
    p.ldh = present(h) ? h->stride_row : 0;
    p.w = weight;
    p.b = bias;
    p.w_f32 = weight_type == GEMM_TYPE_F32;
    p.scale = scale;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.width = width;
    p.eps = eps;
    p.inv_width = 1.0f / float(width);
    p.type = x->type;
    p.out = out_code(y->type, x->type);
    const int es = type_bytes(x->type);
    Places at(p.x, p.ldx, es, rows, width, {weight, bias}, p.w_f32 != 0);
    at.also(p.r, p.ldr, es);
    at.also(p.h, p.ldh, es);
    at.also(p.y, p.ldy, type_bytes(y->type));
    p.vec = at.vec;
    p.shift = !at.vec && at.shift;
    return g16::launch_layer_norm(p, ds->num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_layer_norm_backward_workspace_size(int64_t rows, int64_t width, uint64_t *bytes) {
    if (!sizes_ok(rows, width, 0)) return GEMM_ERR_INVALID_ARG;
    if (bytes) *bytes = uint64_t(std::min<int64_t>(rows, g16::kLayerNormParts)) * uint64_t(width) * 8u;
    return GEMM_OK;
}

gemm_status_t gemm_layer_norm_backward(const gemm_matrix_t *grad, const gemm_matrix_t *h, const void *weight,
                                       int32_t weight_type, const float *mean, const float *rstd,
                                       const gemm_matrix_t *grad_h, const gemm_matrix_t *dx, float *dweight, float *dbias,
                                       int64_t rows, int64_t width, void *workspace, uint64_t workspace_bytes,
                                       gemm_stream_t stream_) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(rows, width, 0) || grad == nullptr || h == nullptr || dx == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!is_c_type(grad->type)) return GEMM_ERR_INVALID_ARG;
    if (weight_type != GEMM_TYPE_F32 && weight_type != grad->type) return GEMM_ERR_INVALID_ARG;
    if (!words_aligned({dweight, dbias})) return GEMM_ERR_INVALID_ARG;
    if (width == 0) return GEMM_OK;
    if (rows > 0) {
        if (grad->data == nullptr || h->data == nullptr || dx->data == nullptr || weight == nullptr || mean == nullptr || rstd == nullptr)
            return GEMM_ERR_INVALID_ARG;
        if (!element_aligned(weight, weight_type) || !words_aligned({mean, rstd})) return GEMM_ERR_INVALID_ARG;
        for (const gemm_matrix_t *m : {grad, h, grad_h, dx}) {
            if (!present(m)) continue;
            if (m->type != grad->type) return GEMM_ERR_INVALID_ARG;
            const gemm_status_t st = check_rows(m, rows, width);
            if (st != GEMM_OK) return st;
        }
    }
    const bool sums = dweight != nullptr || dbias != nullptr;
    uint64_t need = 0;
    if (sums) (void)gemm_layer_norm_backward_workspace_size(rows, width, &need);
    const gemm_status_t st = check_workspace(workspace, workspace_bytes, need, 16);
    if (st != GEMM_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    DeviceState *ds = nullptr;
    const int dev = device_state(&ds);
    if (dev < 0) return GEMM_ERR_CUDA;
    if (rows == 0) {
        for (float *d : {dweight, dbias})
            if (d != nullptr && cudaMemsetAsync(d, 0, size_t(width) * 4u, stream) != cudaSuccess) return GEMM_ERR_CUDA;
        return GEMM_OK;
    }
    g16::LayerNormBackwardArgs p;
    std::memset(&p, 0, sizeof(p));
    p.g = grad->data;
    p.ldg = grad->stride_row;
    p.h = h->data;
    p.ldh = h->stride_row;
    p.dh = present(grad_h) ? grad_h->data : nullptr;
    p.lddh = present(grad_h) ? grad_h->stride_row : 0;
    p.dx = dx->data;
    p.lddx = dx->stride_row;
    p.w = weight;
    p.w_f32 = weight_type == GEMM_TYPE_F32;
    p.mean = mean;
    p.rstd = rstd;
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    p.rows = rows;
    p.width = width;
    p.inv_width = 1.0f / float(width);
    p.type = grad->type;
    const int es = type_bytes(grad->type);
    Places at(p.g, p.ldg, es, rows, width, {weight}, p.w_f32 != 0);
    at.also(p.h, p.ldh, es);
    at.also(p.dh, p.lddh, es);
    at.also(p.dx, p.lddx, es);
    p.vec = at.vec;
    p.shift = !at.vec && at.shift;
    return g16::launch_layer_norm_backward(p, dweight, dbias, dev, ds->num_sms, stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_quantize_rows(const gemm_matrix_t *x, const gemm_matrix_t *q, float *scale, int64_t rows, int64_t width,
                                 gemm_stream_t stream) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(rows, width, 0) || x == nullptr || q == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!is_c_type(x->type) || !is_eight(q->type)) return GEMM_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_OK;
    if (width == 0) {
        if (!words_aligned({scale})) return GEMM_ERR_INVALID_ARG;
        return empty_rows(scale, nullptr, nullptr, rows, 0.0f, reinterpret_cast<cudaStream_t>(stream));
    }
    if (x->data == nullptr || q->data == nullptr || scale == nullptr || !words_aligned({scale})) return GEMM_ERR_INVALID_ARG;
    for (const gemm_matrix_t *m : {x, q}) {
        const gemm_status_t st = check_rows(m, rows, width);
        if (st != GEMM_OK) return st;
    }
    DeviceState *ds = nullptr;
    if (device_state(&ds) < 0) return GEMM_ERR_CUDA;
    g16::QuantizeArgs p;
    std::memset(&p, 0, sizeof(p));
    p.x = x->data;
    p.ldx = x->stride_row;
    p.q = q->data;
    p.ldq = q->stride_row;
    p.scale = scale;
    p.rows = rows;
    p.width = width;
    p.type = x->type;
    p.out = q->type == GEMM_TYPE_I8 ? g16::kOutI8 : g16::kOutE4m3;
    Places at(p.x, p.ldx, type_bytes(x->type), rows, width, {}, false);
    at.also(p.q, p.ldq, 1);
    p.vec = at.vec;
    p.shift = !at.vec && at.shift;
    return g16::launch_quantize_rows(p, ds->num_sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // extern "C"
