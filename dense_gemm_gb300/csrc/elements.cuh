// Elements of rows in registers (sm_103a): vectors as they lie in memory, their values
// in fp32 pairs, rows off 16-byte boundaries, 8-bit floats, and sums and maxima over
// the threads of a row. Used by every kernel that works along rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

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

// VEC consecutive elements as they lie in memory: 16 bytes (32 for fp32) with
// VEC = 8, one element with VEC = 1.
template <typename T, int VEC>
struct Raw {
    static_assert(VEC == 8, "one element, or 16-byte vectors");
    uint4 q[sizeof(T) / 2];
};
template <typename T>
struct Raw<T, 1> {
    T v;
};

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    Raw<T, VEC> r;
    if constexpr (VEC == 1) {
        r.v = *p;
    } else {
#pragma unroll
        for (int i = 0; i < int(sizeof(r) / 16); ++i) r.q[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    return r;
}

// fp32 values in pairs: the arithmetic of a pair is one instruction
// (fma.rn.f32x2 and its like). These kernels spend as many issue slots as the
// memory system leaves them, so VEC = 8 works on 4 pairs; VEC = 1 on one value.
template <int VEC>
struct F32 {
    using E = float2;
    static constexpr int PAIRS = 4;
    E p[PAIRS];
};
template <>
struct F32<1> {
    using E = float;
    static constexpr int PAIRS = 1;
    E p[PAIRS];
};

__device__ __forceinline__ uint64_t bits2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 pair2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float total(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float total(float a) { return a; }

template <int VEC>
__device__ __forceinline__ typename F32<VEC>::E splat(float v) {
    if constexpr (VEC == 8) return make_float2(v, v);
    else return v;
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));  // bf16: the high half of an fp32
}

template <typename T, int VEC>
__device__ __forceinline__ F32<VEC> widen(const Raw<T, VEC> &r) {
    F32<VEC> v;
    if constexpr (VEC == 1) {
        v.p[0] = to_f32<T>(r.v);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v.p[2 * i] = make_float2(__uint_as_float(r.q[i].x), __uint_as_float(r.q[i].y));
            v.p[2 * i + 1] = make_float2(__uint_as_float(r.q[i].z), __uint_as_float(r.q[i].w));
        }
    } else {
        v.p[0] = unpack2<T>(r.q[0].x);
        v.p[1] = unpack2<T>(r.q[0].y);
        v.p[2] = unpack2<T>(r.q[0].z);
        v.p[3] = unpack2<T>(r.q[0].w);
    }
    return v;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T *p, const F32<VEC> &v) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(v.p[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(v.p[2 * i].x, v.p[2 * i].y, v.p[2 * i + 1].x, v.p[2 * i + 1].y);
    } else {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pack2<T>(v.p[0]), pack2<T>(v.p[1]), pack2<T>(v.p[2]), pack2<T>(v.p[3]));
    }
}

// Weights: T or fp32.
template <typename T, int VEC>
__device__ __forceinline__ F32<VEC> load_weight(const void *w, bool w_f32, int64_t at) {
    if (w_f32) return widen<float, VEC>(load_raw<float, VEC>(static_cast<const float *>(w) + at));
    return widen<T, VEC>(load_raw<T, VEC>(static_cast<const T *>(w) + at));
}

// fp32 -> e4m3, nearest even; |v| <= 448 up to rounding, a NaN stays one.
template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const F32<VEC> &v) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(v.p[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(v.p[2 * i], __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(v.p[2 * i + 1], __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// ------------------------------------------------------------------ rows off 16-byte boundaries
// 16-bit rows whose arrays all start at the same place in a granule of 8 elements
// (a contiguous matrix of odd width: every row at another place) are worked on in
// whole granules all the same: `o` elements of the row's first granule are not its
// own, so group i holds the columns 8 i - o ... and the first and last groups are
// cut. A granule with one byte of an allocation lies in its pages, so reading the
// rest of it is safe; its foreign elements are cleared, and never written.
// Element by element, the same rows take 2 to 4 times as long (4096 x 4095 forward
// 65.4 us, so 20.9; backward 66.1 and 36.2).
template <typename T>
__device__ __forceinline__ int place_in_granule(const T *p) {
    return int(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & 7;
}

// Clears the elements outside [lo, hi).
template <typename T>
__device__ __forceinline__ void keep_elems(Raw<T, 8> &r, int lo, int hi) {
    static_assert(sizeof(T) == 2, "eight 16-bit elements");
    uint32_t *w = reinterpret_cast<uint32_t *>(&r.q[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] &= (2 * i >= lo && 2 * i < hi ? 0x0000ffffu : 0u) | (2 * i + 1 >= lo && 2 * i + 1 < hi ? 0xffff0000u : 0u);
}

// Elements s .. s + 7 (0 <= s < 8) of the sixteen in lo and hi.
template <typename T>
__device__ __forceinline__ Raw<T, 8> shift_granules(const Raw<T, 8> &lo, const Raw<T, 8> &hi, int s) {
    const uint32_t x[8] = {lo.q[0].x, lo.q[0].y, lo.q[0].z, lo.q[0].w, hi.q[0].x, hi.q[0].y, hi.q[0].z, hi.q[0].w};
    uint32_t y[6], z[5], o[4];
#pragma unroll
    for (int i = 0; i < 6; ++i) y[i] = (s & 4) ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) z[i] = (s & 2) ? y[i + 1] : y[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (s & 1) ? __funnelshift_r(z[i], z[i + 1], 16) : z[i];
    Raw<T, 8> r;
    r.q[0] = make_uint4(o[0], o[1], o[2], o[3]);
    return r;
}

// Elements at .. at + 7 of w[0 .. width) (16-byte aligned; -8 < at < width), zero
// outside: two granules shifted into one.
template <typename T>
__device__ __forceinline__ Raw<T, 8> load_shifted(const T *w, int at, int width) {
    const int a = at & ~7, s = at & 7;
    Raw<T, 8> lo, hi;
    lo.q[0] = hi.q[0] = make_uint4(0u, 0u, 0u, 0u);
    if (a >= 0) lo = load_raw<T, 8>(w + a);
    if (s != 0 && a + 8 < width) hi = load_raw<T, 8>(w + a + 8);
    Raw<T, 8> r = shift_granules<T>(lo, hi, s);
    if (at + 8 > width) keep_elems<T>(r, 0, width - at);
    return r;
}

__device__ __forceinline__ void store_elems(float *p, const F32<8> &v, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= lo && i < hi) p[i] = i & 1 ? v.p[i / 2].y : v.p[i / 2].x;
}

// v's elements [lo, hi) -> p[lo .. hi): a vector where they are all of them.
template <typename T>
__device__ __forceinline__ void store_some(T *p, const F32<8> &v, int lo, int hi) {
    if (lo <= 0 && hi >= 8) {
        if constexpr (sizeof(T) == 1) store_e4m3<8>(reinterpret_cast<uint8_t *>(p), v);
        else store_f32<T, 8>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < lo || i >= hi) continue;
        F32<1> e;
        e.p[0] = i & 1 ? v.p[i / 2].y : v.p[i / 2].x;
        if constexpr (sizeof(T) == 1) store_e4m3<1>(reinterpret_cast<uint8_t *>(p) + i, e);
        else store_f32<T, 1>(p + i, e);
    }
}

// ------------------------------------------------------------------ row reductions
// A block holds blockDim.y rows of blockDim.x threads each (blockDim.x a
// multiple of 32: a warp never spans two rows). `red`: 32 words, one use between
// two barriers.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Every thread of a row gets the row's sum: each warp's sum goes through shared
// memory, and every warp adds the row's warps' sums by the same tree. One
// barrier, also for rows of one warp where `always` (callers use it to know that
// all threads have left the step before).
template <bool kAlways>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    const int wpr = blockDim.x >> 5;
    if (!kAlways && wpr == 1) return v;
    const int lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (lane == 0) red[base + (threadIdx.x >> 5)] = v;
    __syncthreads();
    if (wpr == 1) return v;
    return warp_sum(lane < wpr ? red[base + lane] : 0.0f);
}

// row_sum<true> of R rows per thread at a time.
template <int R>
__device__ __forceinline__ void rows_sum(float (&v)[R], float (*red)[32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    const int wpr = blockDim.x >> 5, lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) red[r][base + (threadIdx.x >> 5)] = v[r];
    }
    __syncthreads();
    if (wpr == 1) return;
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = lane < wpr ? red[r][base + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// The largest |value|, NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A row's sum and largest value (>= 0 or NaN: their bits are in their order, a
// NaN's above infinity's); one barrier.
__device__ __forceinline__ void row_sum_max(float &v, float &m, float *red, uint32_t *redq) {
    v = warp_sum(v);
    uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu);
    const int wpr = blockDim.x >> 5;
    const int lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (lane == 0) {
        red[base + (threadIdx.x >> 5)] = v;
        redq[base + (threadIdx.x >> 5)] = mb;
    }
    __syncthreads();
    if (wpr > 1) {
        v = warp_sum(lane < wpr ? red[base + lane] : 0.0f);
        mb = __reduce_max_sync(0xffffffffu, lane < wpr ? redq[base + lane] : 0u);
    }
    m = __uint_as_float(mb);
}

// Rows whose largest |y| is below this are stored as zeros with scale 1, as zero
// rows are: their scale would come near the smallest normal number.
constexpr float kQuantTiny = 7.7e-34f;
constexpr float kE4m3Max = 448.0f;
constexpr float kLargest = 3.402823466e38f;

}  // namespace g16
