// Root-mean-square norm with the residual's addition, and its gradients (sm_103a).
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = w h rstd
//   u = h rstd, g = dy w:  dx = rstd (g - u mean(g u)) + dh,  dw = sum_rows dy u
//
// Both directions do a handful of operations per element they move, so DRAM
// bounds them: each row is read once into registers (VEC consecutive elements
// per load, NV loads per thread), reduced over its threads, and written from
// those registers. All sums are fp32, in an order fixed by the launch shape.
#pragma once
#include <cuda_fp8.h>

#include "gemm_kernel.cuh"

namespace g16 {

// ------------------------------------------------------------------ elements
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
    else return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v) {  // round to nearest even
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// A register image of VEC consecutive elements (16 bytes at least with VEC = 8).
template <typename T, int VEC>
struct Raw {
    static_assert(VEC == 1 || VEC == 8, "one element, or 16-byte vectors");
    T v[VEC];
};
template <typename T>
struct alignas(16) Raw<T, 8> {
    T v[8];
};

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    if constexpr (VEC == 1) {
        Raw<T, 1> r;
        r.v[0] = *p;
        return r;
    } else {
        Raw<T, VEC> r;
#pragma unroll
        for (int i = 0; i < int(sizeof(r) / 16); ++i)
            reinterpret_cast<uint4 *>(&r)[i] = reinterpret_cast<const uint4 *>(p)[i];
        return r;
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        Raw<T, VEC> r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < int(sizeof(r) / 16); ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&r)[i];
    }
}

// Weights: T or fp32, VEC of them as fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight(const void *w, bool w_f32, int64_t at, float (&v)[VEC]) {
    if (w_f32) {
        const Raw<float, VEC> r = load_raw<float, VEC>(static_cast<const float *>(w) + at);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = r.v[i];
    } else {
        const Raw<T, VEC> r = load_raw<T, VEC>(static_cast<const T *>(w) + at);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f32<T>(r.v[i]);
    }
}

// fp32 -> e4m3, nearest even; |v| <= 448 up to rounding, a NaN stays one.
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi =
                __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// ------------------------------------------------------------------ row reductions
// A block holds blockDim.y rows of blockDim.x threads each (blockDim.x a
// multiple of 32: a warp never spans two rows). Every thread of a row gets the
// row's sum, its warps' sums added in warp order. `red`: 32 floats, one use per
// call (a second call in the same kernel passes another array).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return v;
    const int w = threadIdx.x >> 5, base = int(threadIdx.y) * wpr;
    if ((threadIdx.x & 31) == 0) red[base + w] = v;
    __syncthreads();
    float s = red[base];
    for (int i = 1; i < wpr; ++i) s += red[base + i];
    return s;
}

// Largest |value| of a row, as bits: the order of the bits of non-negative
// floats is theirs, infinity above every number and a NaN above infinity, so a
// NaN anywhere in the row is the result.
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t *red) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return v;
    const int w = threadIdx.x >> 5, base = int(threadIdx.y) * wpr;
    if ((threadIdx.x & 31) == 0) red[base + w] = v;
    __syncthreads();
    uint32_t m = red[base];
    for (int i = 1; i < wpr; ++i) m = max(m, red[base + i]);
    return m;
}

// Rows whose largest |y| is below this (zero rows among them) are stored as
// zeros with scale 1: their 448 / a would leave fp32's range.
constexpr float kQuantTiny = 7.7e-34f;
constexpr float kE4m3Max = 448.0f;

struct NormParams {
    const void *x, *r;  // r == nullptr: no residual
    const void *w;
    void *y, *h;  // h == nullptr: not stored
    float *scale, *rstd;
    int64_t rows, width;
    int64_t ldx, ldr, ldy, ldh;
    float eps, inv_width;
    int32_t w_f32;
};

__device__ __forceinline__ void quant_factors(uint32_t amax_bits, float &mul, float &scale) {
    const float a = __uint_as_float(amax_bits);
    if (a < kQuantTiny) {
        mul = 0.0f;
        scale = 1.0f;
    } else {  // a NaN makes both NaN
        mul = kE4m3Max / a;
        scale = a * (1.0f / kE4m3Max);
    }
}

// One row per blockDim.x threads, held in registers: element (j * blockDim.x +
// t) * VEC + i of the row is value i of load j of thread t.
template <typename T, int VEC, int NV, bool kQ>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
    __shared__ float red[32];
    __shared__ uint32_t redq[32];
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    griddep_wait();
    griddep_launch_dependents();
    float h[NV][VEC];
    {
        Raw<T, VEC> a[NV], b[NV];
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *r = static_cast<const T *>(p.r) + row * p.ldr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = (int64_t(j) * blockDim.x + threadIdx.x) * VEC;
            if (live && at < p.width) {
                a[j] = load_raw<T, VEC>(x + at);
                if (p.r != nullptr) b[j] = load_raw<T, VEC>(r + at);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = live && (int64_t(j) * blockDim.x + threadIdx.x) * VEC < p.width;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[j][i] = in ? to_f32<T>(a[j].v[i]) : 0.0f;
                if (in && p.r != nullptr) h[j][i] += to_f32<T>(b[j].v[i]);
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(h[j][i], h[j][i], ss);
    if (p.h != nullptr) {
        T *hp = static_cast<T *>(p.h) + row * p.ldh;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = (int64_t(j) * blockDim.x + threadIdx.x) * VEC;
            if (live && at < p.width) store_f32<T, VEC>(hp + at, h[j]);
        }
    }
    const float rstd = rsqrtf(fmaf(row_sum(ss, red), p.inv_width, p.eps));
    if (live && p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t at = (int64_t(j) * blockDim.x + threadIdx.x) * VEC;
        if (live && at < p.width) {
            float w[VEC];
            load_weight<T, VEC>(p.w, p.w_f32 != 0, at, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[j][i] = h[j][i] * rstd * w[i];
                if (kQ) amax = max(amax, __float_as_uint(h[j][i]) & 0x7fffffffu);
            }
            if (!kQ) store_f32<T, VEC>(static_cast<T *>(p.y) + row * p.ldy + at, h[j]);
        }
    }
    if constexpr (kQ) {
        float mul, scale;
        quant_factors(row_max_bits(amax, redq), mul, scale);
        if (!live) return;
        if (threadIdx.x == 0) p.scale[row] = scale;
        uint8_t *q = static_cast<uint8_t *>(p.y) + row * p.ldy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = (int64_t(j) * blockDim.x + threadIdx.x) * VEC;
            if (at < p.width) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[j][i] *= mul;
                store_e4m3<VEC>(q + at, h[j]);
            }
        }
    }
}

// Rows longer than the register form holds: one block per row, which reads its
// row once per pass (sum, with 8 bits the maximum, store); a thread re-reads
// only what it wrote itself, so h may be x or r.
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const NormParams p, int32_t quant) {
    __shared__ float red[32];
    __shared__ uint32_t redq[32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = p.r != nullptr ? static_cast<const T *>(p.r) + row * p.ldr : nullptr;
    auto sum = [&](int64_t at) { return to_f32<T>(x[at]) + (r != nullptr ? to_f32<T>(r[at]) : 0.0f); };
    float ss = 0.0f;
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float h = sum(at);
        ss = fmaf(h, h, ss);
    }
    const float rstd = rsqrtf(fmaf(row_sum(ss, red), p.inv_width, p.eps));
    if (p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
    float mul = 1.0f, scale = 1.0f;
    if (quant) {
        uint32_t amax = 0;
        for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
            float w[1];
            load_weight<T, 1>(p.w, p.w_f32 != 0, at, w);
            amax = max(amax, __float_as_uint(sum(at) * rstd * w[0]) & 0x7fffffffu);
        }
        quant_factors(row_max_bits(amax, redq), mul, scale);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        float w[1];
        load_weight<T, 1>(p.w, p.w_f32 != 0, at, w);
        const float h = sum(at);
        float y[1] = {h * rstd * w[0]};
        if (p.h != nullptr) static_cast<T *>(p.h)[row * p.ldh + at] = from_f32<T>(h);
        if (quant) {
            y[0] *= mul;
            store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.ldy + at, y);
        } else {
            static_cast<T *>(p.y)[row * p.ldy + at] = from_f32<T>(y[0]);
        }
    }
}

// ------------------------------------------------------------------ backward
struct NormBackwardParams {
    const void *g, *h, *dh;  // dh == nullptr: none
    const void *w;
    const float *rstd;
    void *dx;
    float *partial;  // [gridDim.x][width] column sums of this block's rows; nullptr: dweight not asked for
    int64_t rows, width;
    int64_t ldg, ldh, lddh, lddx;
    float inv_width;
    int32_t w_f32;
};

// Rows blockIdx.x * blockDim.y + threadIdx.y, then every gridDim.x * blockDim.y
// further on: a thread keeps its columns, so their dweight sums stay in its
// registers and each block writes one row of partial sums at its end. The next
// row's loads are issued before this row's reduction, whose barrier would
// otherwise leave the block with nothing in flight.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024) rms_norm_backward_kernel(const NormBackwardParams p) {
    __shared__ float red[2][32];
    extern __shared__ float dw_rows[];  // blockDim.y > 1: [blockDim.y][blockDim.x * VEC * NV]
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    // the block's rows advance together, so that the barriers below are met by all
    const int64_t first = int64_t(blockIdx.x) * blockDim.y;
    float w[NV][VEC], dw[NV][VEC];
    Raw<T, VEC> rg[NV], rh[NV], rd[NV];
    float rstd = 0.0f;
    auto at_of = [&](int j) { return (int64_t(j) * blockDim.x + threadIdx.x) * VEC; };
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
        rstd = p.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (at_of(j) >= p.width) continue;
            rg[j] = load_raw<T, VEC>(static_cast<const T *>(p.g) + row * p.ldg + at_of(j));
            rh[j] = load_raw<T, VEC>(static_cast<const T *>(p.h) + row * p.ldh + at_of(j));
            if (p.dh != nullptr) rd[j] = load_raw<T, VEC>(static_cast<const T *>(p.dh) + row * p.lddh + at_of(j));
        }
    };
    fetch(first + threadIdx.y);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = dw[j][i] = 0.0f;
        if (at_of(j) < p.width) load_weight<T, VEC>(p.w, p.w_f32 != 0, at_of(j), w[j]);
    }
    int flip = 0;
    for (int64_t base = first; base < p.rows; base += step, flip ^= 1) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < p.rows;
        const float rs = rstd;
        float g[NV][VEC], u[NV][VEC], d[NV][VEC];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = live && at_of(j) < p.width;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float dy = in ? to_f32<T>(rg[j].v[i]) : 0.0f;
                u[j][i] = in ? to_f32<T>(rh[j].v[i]) * rs : 0.0f;
                d[j][i] = in && p.dh != nullptr ? to_f32<T>(rd[j].v[i]) : 0.0f;
                g[j][i] = dy * w[j][i];
                dw[j][i] = fmaf(dy, u[j][i], dw[j][i]);
                dot = fmaf(g[j][i], u[j][i], dot);
            }
        }
        fetch(row + step);
        const float m = row_sum(dot, red[flip]) * p.inv_width;
        if (live) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (at_of(j) >= p.width) continue;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = fmaf(rs, fmaf(-u[j][i], m, g[j][i]), d[j][i]);
                store_f32<T, VEC>(static_cast<T *>(p.dx) + row * p.lddx + at_of(j), o);
            }
        }
    }
    if (p.partial == nullptr) return;
    if (blockDim.y > 1) {
        const int span = blockDim.x * VEC * NV;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) dw_rows[int(threadIdx.y) * span + int(at_of(j)) + i] = dw[j][i];
        __syncthreads();
        const int t = threadIdx.y * blockDim.x + threadIdx.x;
        for (int c = t; c < span && c < p.width; c += blockDim.x * blockDim.y) {
            float s = dw_rows[c];
            for (int y = 1; y < int(blockDim.y); ++y) s += dw_rows[y * span + c];
            p.partial[int64_t(blockIdx.x) * p.width + c] = s;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (at_of(j) >= p.width) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) p.partial[int64_t(blockIdx.x) * p.width + at_of(j) + i] = dw[j][i];
    }
}

// Rows longer than the register form holds: dx with one block per row (two
// passes over it), dweight's column sums by another kernel.
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_backward_long_kernel(const NormBackwardParams p) {
    __shared__ float red[32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *g = static_cast<const T *>(p.g) + row * p.ldg, *h = static_cast<const T *>(p.h) + row * p.ldh;
    const T *dh = p.dh != nullptr ? static_cast<const T *>(p.dh) + row * p.lddh : nullptr;
    const float rs = p.rstd[row];
    float dot = 0.0f;
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        float w[1];
        load_weight<T, 1>(p.w, p.w_f32 != 0, at, w);
        dot = fmaf(to_f32<T>(g[at]) * w[0], to_f32<T>(h[at]) * rs, dot);
    }
    const float m = row_sum(dot, red) * p.inv_width;
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        float w[1];
        load_weight<T, 1>(p.w, p.w_f32 != 0, at, w);
        const float u = to_f32<T>(h[at]) * rs;
        const float d = dh != nullptr ? to_f32<T>(dh[at]) : 0.0f;
        static_cast<T *>(p.dx)[row * p.lddx + at] = from_f32<T>(fmaf(rs, fmaf(-u, m, to_f32<T>(g[at]) * w[0]), d));
    }
}

template <typename T>
__global__ void __launch_bounds__(256) rms_norm_dweight_long_kernel(const NormBackwardParams p, int64_t rows_per_block) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t col = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t r0 = int64_t(blockIdx.y) * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < p.rows ? r0 + rows_per_block : p.rows;
    if (col >= p.width) return;
    float s = 0.0f;
    for (int64_t row = r0; row < r1; ++row)
        s = fmaf(to_f32<T>(static_cast<const T *>(p.g)[row * p.ldg + col]),
                 to_f32<T>(static_cast<const T *>(p.h)[row * p.ldh + col]) * p.rstd[row], s);
    p.partial[int64_t(blockIdx.y) * p.width + col] = s;
}

// out[c] = sum of partial[0..parts)[c]: 32 columns per block, blockDim.y threads
// each add every blockDim.y-th row, then the first adds theirs in order.
constexpr int kPartGroups = 32;
__global__ void __launch_bounds__(32 * kPartGroups) sum_partials_kernel(const float *__restrict__ partial,
                                                                        float *__restrict__ out, int64_t parts,
                                                                        int64_t width) {
    __shared__ float s[kPartGroups][33];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.0f;
    if (col < width) {
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < parts; r += kPartGroups) v += partial[r * width + col];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || col >= width) return;
    for (int g = 1; g < kPartGroups; ++g) v += s[g][threadIdx.x];
    out[col] = v;
}

}  // namespace g16
