// Layer norm with the residual's addition, its gradients, and rows in 8 bits (sm_103a).
//
//   h = x + r,  mean, var over the row,  rstd = 1 / sqrt(var + eps),  y = w (h - mean) rstd + b
//   u = (h - mean) rstd, g = dy w:  dx = rstd (g - mean(g) - u mean(g u)) + dh,
//                                   dw = sum_rows dy u,  db = sum_rows dy
//   q = round(x TOP / a), scale = a / TOP,  a = max|x| of the row, TOP 448 (e4m3) or 127 (int8)
//
// A dozen operations per element at most: the floor of all of them is DRAM's, so every row is
// read once into registers or shared memory and written from there. They come near it where rows are
// many and some thousand elements wide; elsewhere what a row does in series (loads, sums over its
// threads, store) counts, with too few loads in flight meanwhile: neither DRAM nor the issue slots are
// full. The variance is summed from the centred values: the difference of the mean square and the squared
// mean loses what a row's mean has more digits than its deviation; a mean that is large beside
// it is corrected by their own sum (RowMean). All sums are fp32, in an order that the sizes fix.
#include "ops_rows.h"

#include <algorithm>
#include <atomic>
#include <utility>

#include "elements.cuh"
#include "rows_check.cuh"

namespace g16 {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// As the other kernels of the library: programmatic stream serialization allowed.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// Raises a kernel's shared-memory limit, once per device.
template <auto Kernel>
cudaError_t allow_smem(int dev, int bytes) {
    static std::atomic<uint64_t> raised{0};  // one bit per device
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (raised.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) (void)cudaGetLastError();
    else raised.fetch_or(bit, std::memory_order_release);
    return e;
}

// ------------------------------------------------------------------ 8 bits with a scale per row
template <int OUT>
constexpr float kTop = OUT == kOutI8 ? 127.0f : kE4m3Max;

// A row's factor and scale from a = max|y|. An infinity or a NaN makes the scale NaN,
// and with it every value; the bytes are NaNs in e4m3 and zeros in int8.
template <int OUT>
__device__ __forceinline__ void row_factor(float a, float &mul, float &scale) {
    if (a < kQuantTiny) {
        mul = 0.0f;
        scale = 1.0f;
    } else if (!(a <= kLargest)) {
        mul = scale = __int_as_float(0x7fffffff);  // NaN
    } else {
        mul = kTop<OUT> / a;
        scale = a * (1.0f / kTop<OUT>);
    }
}

// What t / a has beyond its fp32 value `mul`: x mul + x rest is x t / a within 2^-47 of it, so
// that a value of 16 bits that lies on a rounding's edge is found there and goes to the even
// side. (mul alone is up to 2^-24 off, and of 4096 x 16384 bf16 values 3 in 10,000 went to the
// other side; it took 31.6 us to e4m3 and 32.0 to int8, this 32.0 and 33.1. With the rest from a
// division 37.8 and 39.2.) A row whose mul is 0 or NaN has no rest.
template <int OUT>
__device__ __forceinline__ float factor_rest(float a, float mul) {
    return mul > 0.0f ? fmaf(-mul, a, kTop<OUT>) * (mul * (1.0f / kTop<OUT>)) : 0.0f;  // mul / t: near enough to 1 / a
}

// fp32 -> int8, nearest even: 1.5 2^23 + v, |v| <= 127 up to rounding, has v's two's
// complement in its last byte, so that the rounding and the conversion are one addition
// (4096 x 16384 with a look for NaNs at each value 36.8 us, without 33.3), and where the row's
// factor is one number (a norm's y) one multiply-add with it.
constexpr float kI8Shift = 12582912.0f;
__device__ __forceinline__ uint32_t pack_i8x4(float2 a, float2 b) {
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

template <int OUT, typename T>
using Stored = std::conditional_t<OUT == kOutSame, T, uint8_t>;

// Eight values times the row's factor -> p, those of [lo, hi). kRest: the factor is mul + rest.
// `zeros`: an int8 row whose scale is NaN.
template <typename T, int OUT, bool kRest = false>
__device__ __forceinline__ void store_out(Stored<OUT, T> *p, F32<8> v, float mul, bool zeros, int lo, int hi, float rest = 0.0f) {
    if constexpr (kRest) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = fma2(v.p[i], splat<8>(mul), mul2(v.p[i], splat<8>(rest)));
    }
    if constexpr (OUT == kOutI8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.p[i] = kRest ? add2(v.p[i], splat<8>(kI8Shift)) : fma2(v.p[i], splat<8>(mul), splat<8>(kI8Shift));
        uint2 w = make_uint2(pack_i8x4(v.p[0], v.p[1]), pack_i8x4(v.p[2], v.p[3]));
        if (zeros) w = make_uint2(0u, 0u);
        if (lo <= 0 && hi >= 8) {
            *reinterpret_cast<uint2 *>(p) = w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= lo && i < hi) p[i] = uint8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    } else {
        if constexpr (OUT == kOutE4m3 && !kRest) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v.p[i] = mul2(v.p[i], splat<8>(mul));
        }
        store_some<Stored<OUT, T>>(p, v, lo, hi);
    }
}
template <typename T>
__device__ __forceinline__ void store_same(T *p, const F32<8> &v, int lo, int hi) {
    store_out<T, kOutSame>(p, v, 1.0f, false, lo, hi);
}
template <typename T, int OUT>
__device__ __forceinline__ void store_one(void *p, int64_t at, float v, float mul, bool zeros) {
    if constexpr (OUT == kOutI8) static_cast<uint8_t *>(p)[at] = zeros ? uint8_t(0) : uint8_t(__float_as_uint(fmaf(v, mul, kI8Shift)));
    else if constexpr (OUT == kOutE4m3) static_cast<uint8_t *>(p)[at] = __nv_cvt_float_to_fp8(v * mul, __NV_SATFINITE, __NV_E4M3);
    else static_cast<T *>(p)[at] = from_f32<T>(v);
}

// row_sum<false> with a barrier of the row's own threads: rows side by side in a block need not all take it.
__device__ __forceinline__ float own_row_sum(float v, float *red) {
    v = warp_sum(v);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return v;
    const int lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (lane == 0) red[base + (threadIdx.x >> 5)] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
    return warp_sum(lane < wpr ? red[base + lane] : 0.0f);
}

// Every thread of a row gets the row's largest m (>= 0 or NaN: their bits are in their
// order, a NaN's above infinity's); one barrier.
__device__ __forceinline__ float row_max(float m, uint32_t *red) {
    uint32_t b = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu);
    const int wpr = blockDim.x >> 5;
    if (wpr == 1) return __uint_as_float(b);
    const int lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (lane == 0) red[base + (threadIdx.x >> 5)] = b;
    __syncthreads();
    return __uint_as_float(__reduce_max_sync(0xffffffffu, lane < wpr ? red[base + lane] : 0u));
}

__device__ __forceinline__ float largest(const F32<8> &v, float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_nan(max_nan(m, fabsf(v.p[i].x)), fabsf(v.p[i].y));
    return m;
}

// ------------------------------------------------------------------ rows in registers
// NV loads of 8 elements per thread; element (j blockDim.x + t) 8 + i of the row is value
// i of load j of thread t. kShift: rows off 16-byte boundaries, their first element `o`
// into a granule; elements of a granule that are not the row's are zero.
template <typename T, int NV, bool kShift>
struct Row {
    int o, width;
    bool live;
    __device__ __forceinline__ Row(const T *first, int width_, bool live_)
        : o(kShift && live_ ? place_in_granule(first) : 0), width(width_), live(live_) {}
    __device__ __forceinline__ int at(int j) const { return (j * int(blockDim.x) + int(threadIdx.x)) * 8 - o; }
    __device__ __forceinline__ bool has(int j) const { return live && at(j) < width; }
    __device__ __forceinline__ bool cut(int j) const { return kShift && (at(j) < 0 || at(j) + 8 > width); }
    __device__ __forceinline__ int lo(int j) const { return kShift ? -at(j) : 0; }
    __device__ __forceinline__ int hi(int j) const { return kShift ? width - at(j) : 8; }
    // (checks) load j's granule has an element of the row, is all the row's unless shifted, and lies at `p` on
    // the boundary that its elements' size asks for
    __device__ __forceinline__ bool ok(int j, const void *p, int es) const {
        return live && at(j) > -8 && at(j) < width && (kShift || (at(j) >= 0 && at(j) + 8 <= width)) &&
               (reinterpret_cast<uintptr_t>(p) & uintptr_t(es == 1 ? 7 : 15)) == 0;
    }
    __device__ __forceinline__ void keep(Raw<T, 8> &r, int j) const {
        if constexpr (kShift) {
            if (cut(j)) keep_elems<T>(r, lo(j), hi(j));
        }
    }
    // a vector that starts with the row's columns: weights
    __device__ __forceinline__ Raw<T, 8> column(const void *w, int j) const {
        if constexpr (kShift) return load_shifted<T>(static_cast<const T *>(w), at(j), width);
        else return load_raw<T, 8>(static_cast<const T *>(w) + at(j));
    }
    __device__ __forceinline__ F32<8> column(const void *w, bool f32, int j) const {
        if (!kShift && f32) return widen<float, 8>(load_raw<float, 8>(static_cast<const float *>(w) + at(j)));
        return widen<T, 8>(column(w, j));
    }
};

__device__ __forceinline__ void clear_outside(F32<8> &v, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (2 * i < lo || 2 * i >= hi) v.p[i].x = 0.0f;
        if (2 * i + 1 < lo || 2 * i + 1 >= hi) v.p[i].y = 0.0f;
    }
}

// A row's mean and variance. m1 = sum / width is as many roundings off as the sum has: none or few for
// values of 16 bits, units of m1's last place where the mean is large beside the deviation. Past four
// deviations c = h - m1 is exact or nearly so, the mean of c is what m1 lacks, and the variance is that
// of the values less the two. Without it a row of equal values keeps some units of its mean's last
// place for c, which 1 / sqrt(eps) multiplies (eps = 1e-12: y = b +- w). What the correction leaves of
// the variance below the sums' own rounding is 0. (Without it 8192 x 4096 43.4 us, so 44.5, 4096 x 8192 to
// 8 bits 39.0 and 39.8; rows that take it, 8192 x 4096 without a residual, 33.5 and 39.6. For every row,
// with one barrier for both sums, 44.7, 40.6 and 35.7.)
__device__ __forceinline__ float first_mean(float sum, float width, float inv_width) {
    const float m = sum * inv_width;
    const float r = fmaf(fmaf(-m, width, sum), inv_width, m);  // sum / width, rounded once
    return r - r == 0.0f ? r : m;
}
struct RowMean {
    float mean, var, less;  // c - less is h - mean
    __device__ __forceinline__ RowMean(float m1, float square) : mean(m1), var(square), less(0.0f) {}
    __device__ __forceinline__ bool rough() const { return __builtin_expect(var < 0.0625f * mean * mean, 0); }
    __device__ __forceinline__ void correct(float more) {  // by the mean of c
        const float m1 = mean, square = var;
        mean = m1 + more;
        less = mean - m1;
        var = fmaf(less, less - 2.0f * more, square);
        if (var < square * 0x1p-16f) var = 0.0f;
    }
};

// Many rows: 4096 x 8192 bf16 with residual to 8 bits 235 MB in 42.0 us (5.6 TB/s), 8192 x 4096 268 MB
// in 46.1 (5.8), DRAM and the issue slots each three fifths busy: the blocks on an SM (64 registers a
// thread) have too few loads in flight while others sum. Few: the chain load - sums - store
// (1 x 4096 2.1 us, 1000 x 5000 10.4 for 5.9 of DRAM). Loads that pass L1 for x and r, to leave it to the
// weights, were 2 to 4 % slower.
template <typename T, int NV, int OUT, bool kShift>
__global__ void __launch_bounds__(1024) layer_norm_kernel(const LayerNormArgs p) {
    __shared__ float red[3][32];
    __shared__ uint32_t redq[32];
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const Row<T, NV, kShift> a(x, int(p.width), row < p.rows);
    constexpr bool kEarly = NV <= 2;  // weights on their way before the sums; four loads' would not fit the registers
    const bool early = kEarly && !p.w_f32;
    F32<8> t[NV];
    Raw<T, 8> w[NV], b[NV];
    {
        Raw<T, 8> rx[NV], rr[NV];
        const T *r = static_cast<const T *>(p.r) + row * p.ldr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!a.has(j) || !G16_CHECK(row < p.rows && a.ok(j, x + a.at(j), sizeof(T)))) continue;
            rx[j] = load_raw<T, 8>(x + a.at(j));
            if (p.r != nullptr && G16_CHECK(a.ok(j, r + a.at(j), sizeof(T)))) rr[j] = load_raw<T, 8>(r + a.at(j));
        }
        if constexpr (kEarly) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!a.has(j) || !early) continue;
                w[j] = a.column(p.w, j);
                if (p.b != nullptr) b[j] = a.column(p.b, j);
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!a.has(j)) continue;
            a.keep(rx[j], j);
            t[j] = widen<T, 8>(rx[j]);
            if (p.r == nullptr) continue;
            a.keep(rr[j], j);
            const F32<8> f = widen<T, 8>(rr[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = add2(t[j].p[i], f.p[i]);
        }
    }
    float2 sum = splat<8>(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!a.has(j)) continue;
        T *h = static_cast<T *>(p.h) + row * p.ldh + a.at(j);
        if (p.h != nullptr && G16_CHECK(a.ok(j, h, sizeof(T)))) store_same<T>(h, t[j], a.lo(j), a.hi(j));
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = add2(sum, t[j].p[i]);
    }
    const float m1 = first_mean(row_sum<false>(total(sum), red[0]), float(a.width), p.inv_width);
    float2 ss = splat<8>(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!a.has(j)) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j].p[i] = add2(t[j].p[i], splat<8>(-m1));
        if (a.cut(j)) clear_outside(t[j], a.lo(j), a.hi(j));
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(t[j].p[i], t[j].p[i], ss);
    }
    RowMean m(m1, row_sum<false>(total(ss), red[1]) * p.inv_width);
    if (m.rough()) {
        sum = splat<8>(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!a.has(j)) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = add2(sum, t[j].p[i]);
        }
        m.correct(own_row_sum(total(sum), red[2]) * p.inv_width);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!a.has(j)) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j].p[i] = add2(t[j].p[i], splat<8>(-m.less));
        }
    }
    const float mean = m.mean, rstd = rsqrtf(m.var + p.eps);
    float top = 0.0f;
    Stored<OUT, T> *y = static_cast<Stored<OUT, T> *>(p.y) + row * p.ldy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!a.has(j)) continue;
        const F32<8> fw = early ? widen<T, 8>(w[j]) : a.column(p.w, p.w_f32 != 0, j);
        F32<8> fb;
        if (p.b != nullptr) fb = early ? widen<T, 8>(b[j]) : a.column(p.b, p.w_f32 != 0, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = mul2(t[j].p[i], splat<8>(rstd));
            t[j].p[i] = p.b != nullptr ? fma2(u, fw.p[i], fb.p[i]) : mul2(u, fw.p[i]);
        }
        if constexpr (OUT != kOutSame) top = largest(t[j], top);
        else if (G16_CHECK(a.ok(j, y + a.at(j), sizeof(*y)))) store_same<T>(y + a.at(j), t[j], a.lo(j), a.hi(j));
    }
    if (a.live && threadIdx.x == 0) {
        if (p.mean != nullptr) p.mean[row] = mean;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    if constexpr (OUT != kOutSame) {
        float mul, scale;
        row_factor<OUT>(row_max(top, redq), mul, scale);
        if (a.live && threadIdx.x == 0) p.scale[row] = scale;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (a.has(j) && G16_CHECK(a.ok(j, y + a.at(j), sizeof(*y))))
                store_out<T, OUT>(y + a.at(j), t[j], mul, scale != scale, a.lo(j), a.hi(j));
        }
    }
}

// Rows that the register form does not take: longer ones, arrays that disagree on their
// place in a granule, fp32 off 16-byte boundaries. One block per row, element by element;
// the row's sums h are kept in shared memory where they fit (`cached`), else made again
// in each pass. A thread re-reads only what it wrote itself, and h is stored in the last
// pass, so h may be x or r.
template <typename T, int OUT>
__global__ void __launch_bounds__(1024) layer_norm_any_kernel(const LayerNormArgs p, int32_t cached) {
    extern __shared__ float kept[];
    __shared__ float red[3][32];
    __shared__ uint32_t redq[32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = p.r != nullptr ? static_cast<const T *>(p.r) + row * p.ldr : nullptr;
    auto made = [&](int64_t at) { return to_f32<T>(x[at]) + (r != nullptr ? to_f32<T>(r[at]) : 0.0f); };
    auto value = [&](int64_t at) { return cached ? kept[at] : made(at); };
    float s = 0.0f;
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float h = made(at);
        if (cached && G16_CHECK(smem_window_ok(smem_addr(kept + at), 4))) kept[at] = h;
        s += h;
    }
    const float m1 = first_mean(row_sum<false>(s, red[0]), float(p.width), p.inv_width);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float c = value(at) - m1;
        s1 += c;
        s2 = fmaf(c, c, s2);
    }
    RowMean m(m1, row_sum<false>(s2, red[1]) * p.inv_width);
    if (m.rough()) m.correct(own_row_sum(s1, red[2]) * p.inv_width);
    const float mean = m.mean, rstd = rsqrtf(m.var + p.eps);
    auto result = [&](float h, int64_t at) {
        const float w = load_weight<T, 1>(p.w, p.w_f32 != 0, at).p[0], u = (h - mean) * rstd;
        return p.b != nullptr ? fmaf(u, w, load_weight<T, 1>(p.b, p.w_f32 != 0, at).p[0]) : u * w;
    };
    if (threadIdx.x == 0) {
        if (p.mean != nullptr) p.mean[row] = mean;
        if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    float mul = 1.0f, scale = 1.0f;
    if constexpr (OUT != kOutSame) {
        float top = 0.0f;
#pragma unroll 4
        for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) top = max_nan(top, fabsf(result(value(at), at)));
        row_factor<OUT>(row_max(top, redq), mul, scale);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float h = value(at);
        const float y = result(h, at);
        if (p.h != nullptr) static_cast<T *>(p.h)[row * p.ldh + at] = from_f32<T>(h);
        store_one<T, OUT>(p.y, row * p.ldy + at, y, mul, scale != scale);
    }
}

// ------------------------------------------------------------------ rows in 8 bits
// One pass: the row stays in registers between its maximum and its store. 4096 x 16384 bf16 takes
// 33.4 us (201 MB, 6.0 TB/s, nine tenths of a copy's rate), to int8 34.7; 999 x 5001 fp16 5.4 us. 40
// registers: three blocks of 512 threads on an SM (4096 x 16384 to int8 38.9 us with 42).
template <typename T, int NV, int OUT, bool kShift>
__global__ void __maxnreg__(sizeof(T) == 2 ? 40 : 64) quantize_rows_kernel(const QuantizeArgs p) {
    __shared__ uint32_t redq[32];
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    griddep_wait();
    griddep_launch_dependents();
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const Row<T, NV, kShift> a(x, int(p.width), row < p.rows);
    Raw<T, 8> rx[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (a.has(j) && G16_CHECK(row < p.rows && a.ok(j, x + a.at(j), sizeof(T)))) rx[j] = load_raw<T, 8>(x + a.at(j));
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!a.has(j)) continue;
        a.keep(rx[j], j);
        top = largest(widen<T, 8>(rx[j]), top);
    }
    float mul, scale;
    top = row_max(top, redq);
    row_factor<OUT>(top, mul, scale);
    const float rest = factor_rest<OUT>(top, mul);
    if (a.live && threadIdx.x == 0) p.scale[row] = scale;
    uint8_t *q = static_cast<uint8_t *>(p.q) + row * p.ldq;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!a.has(j) || !G16_CHECK(a.ok(j, q + a.at(j), 1))) continue;
        store_out<T, OUT, true>(q + a.at(j), widen<T, 8>(rx[j]), mul, scale != scale, a.lo(j), a.hi(j), rest);
    }
}

template <typename T, int OUT>
__global__ void __launch_bounds__(1024) quantize_any_kernel(const QuantizeArgs p, int32_t cached) {
    extern __shared__ float kept[];
    __shared__ uint32_t redq[32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    float top = 0.0f, mul, scale;
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float v = to_f32<T>(x[at]);
        if (cached && G16_CHECK(smem_window_ok(smem_addr(kept + at), 4))) kept[at] = v;
        top = max_nan(top, fabsf(v));
    }
    top = row_max(top, redq);
    row_factor<OUT>(top, mul, scale);
    const float rest = factor_rest<OUT>(top, mul);
    if (threadIdx.x == 0) p.scale[row] = scale;
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float v = cached ? kept[at] : to_f32<T>(x[at]);
        store_one<T, OUT>(p.q, row * p.ldq + at, fmaf(v, mul, v * rest), 1.0f, scale != scale);
    }
}

// ------------------------------------------------------------------ gradients
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src) {
    if (!G16_CHECK(((dst | uint32_t(reinterpret_cast<uintptr_t>(src))) & 15u) == 0 && smem_window_ok(dst, 16))) return;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kBackThreads = 512;  // of a block at most: 128 registers each

// (checks) column `col` of part `part` lies in the workspace
[[maybe_unused]] __device__ __forceinline__ bool part_ok(const LayerNormBackwardArgs &p, int64_t part, int64_t col) {
    return p.partial != nullptr && part < p.rows && part < kLayerNormParts && col >= 0 && col < p.width;
}

// rows_sum for rows side by side in a block that do not wait for one another: a barrier
// of the row's own threads, none for a row of one warp.
template <int N>
__device__ __forceinline__ void own_rows_sum(float (&v)[N], float (*red)[32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < N; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    const int wpr = blockDim.x >> 5, lane = threadIdx.x & 31, base = int(threadIdx.y) * wpr;
    if (wpr == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < N; ++r) red[r][base + (threadIdx.x >> 5)] = v[r];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] = lane < wpr ? red[r][base + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < N; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// The persistent form: a block of up to 512 threads walks over the rows, several side by side where
// they are short; its threads keep their columns and the sums of dweight and dbias over
// them, and the rows of the next STAGES - 1 steps are on their way into shared memory. A
// thread copies what it will itself read, so that a step waits for the thread's own
// copies only; the one barrier of a step is that of the two row sums, for R rows at a time.
// 8192 x 4096 bf16 with grad_h 268 MB in 46 us (5.8 TB/s), 50.5 with the partial sums' launch: DRAM two
// thirds, issue slots 56 % busy, one block of 16 warps on an SM. 4096 x 8192 53.4. Twice DRAM's time at
// 8192 x 1024 (20.4 us for 9.9: one load per thread, a barrier for 128 of them) and 2048 x 16384 (79 for
// 39.6: one row and one step ahead), more where rows are few (513 x 4095 fp16 13.4 for 1.9).
// kShift: rows off 16-byte boundaries. A thread's rows are then a multiple of 8 rows apart
// (the grid is a multiple of 8), so that all of them start at the same place in a granule
// and the thread keeps its columns.
template <typename T, int NV, int R, int STAGES, bool kShift>
__global__ void __launch_bounds__(kBackThreads) layer_norm_backward_rows_kernel(const LayerNormBackwardArgs p) {
    constexpr int G = int(sizeof(Raw<T, 8>)) / 16;          // granules of a load
    constexpr uint32_t LINE = uint32_t(kBackThreads) * 16u;  // one granule of every thread
    constexpr uint32_t ARRAY = R * NV * G * LINE, STAGE = 3 * ARRAY;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][2 * R][32];
    const int tid = int(threadIdx.y * blockDim.x + threadIdx.x);
    griddep_wait();
    griddep_launch_dependents();
    const int64_t base0 = int64_t(blockIdx.x) * int(blockDim.y) * (kShift ? 1 : R);  // the block's first row
    const int64_t first = base0 + int(threadIdx.y) * (kShift ? 1 : R);
    const int64_t step = int64_t(gridDim.x) * int(blockDim.y) * R;
    const int64_t apart = kShift ? int64_t(gridDim.x) * blockDim.y : 1;  // rows between a thread's R rows
    const bool has_d = p.dh != nullptr;
    const Row<T, NV, kShift> a(static_cast<const T *>(p.g) + first * p.ldg, int(p.width), first < p.rows);
    bool has[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) has[j] = a.has(j);
    // this thread's first element of the rows to be fetched and written next; the others by offsets in bytes
    const char *gp = reinterpret_cast<const char *>(static_cast<const T *>(p.g) + first * p.ldg + a.at(0));
    const char *hp = reinterpret_cast<const char *>(static_cast<const T *>(p.h) + first * p.ldh + a.at(0));
    const char *dp = reinterpret_cast<const char *>(static_cast<const T *>(p.dh) + first * p.lddh + a.at(0));
    char *xp = reinterpret_cast<char *>(static_cast<T *>(p.dx) + first * p.lddx + a.at(0));
    constexpr int64_t E = int64_t(sizeof(T));
    const int64_t g_step = step * p.ldg * E, h_step = step * p.ldh * E, d_step = step * p.lddh * E, x_step = step * p.lddx * E;
    const int64_t g_row = apart * p.ldg * E, h_row = apart * p.ldh * E, d_row = apart * p.lddh * E, x_row = apart * p.lddx * E;
    const uint32_t jump = blockDim.x * 16u * G;  // bytes between a thread's loads
    const uint32_t mine = smem_addr(ring) + uint32_t(tid) * 16u;
    // (checks) a stepped address is that of load j of `row`, which exists
    [[maybe_unused]] auto at_row = [&](const char *stepped, const void *base, int64_t ld, int64_t row, int j) {
        const T *direct = static_cast<const T *>(base) + row * ld + a.at(j);
        return row >= 0 && row < p.rows && stepped == reinterpret_cast<const char *>(direct) && a.ok(j, direct, sizeof(T));
    };
    // rows row, row + apart, ... -> the slot at `to`; on to the next step's
    auto fetch = [&](int64_t row, uint32_t to) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row + r * apart >= p.rows) break;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!has[j] || !G16_CHECK(at_row(gp + r * g_row + j * jump, p.g, p.ldg, row + r * apart, j) &&
                                          at_row(hp + r * h_row + j * jump, p.h, p.ldh, row + r * apart, j) &&
                                          (!has_d || at_row(dp + r * d_row + j * jump, p.dh, p.lddh, row + r * apart, j))))
                    continue;
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const uint32_t at = to + uint32_t((r * NV + j) * G + k) * LINE;
                    copy16_async(at, gp + r * g_row + j * jump + 16 * k);
                    copy16_async(at + ARRAY, hp + r * h_row + j * jump + 16 * k);
                    if (has_d) copy16_async(at + 2 * ARRAY, dp + r * d_row + j * jump + 16 * k);
                }
            }
        }
        copies_commit();
        gp += g_step;
        hp += h_step;
        dp += d_step;
    };
    auto values = [&](uint32_t at, int j) {
        Raw<T, 8> v = {};
#pragma unroll
        for (int k = 0; k < G; ++k)
            if (G16_CHECK(smem_window_ok(at + k * LINE, 16))) asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.q[k].x), "=r"(v.q[k].y), "=r"(v.q[k].z), "=r"(v.q[k].w)
                         : "r"(at + k * LINE)
                         : "memory");
        a.keep(v, j);
        return widen<T, 8>(v);
    };
    F32<8> dw[NV], db[NV];
    // a weight of T's type; fp32 weights, and those of four loads per thread, whose registers
    // the sums need, are read again for each row
    constexpr bool kKeep = NV < 4;
    Raw<T, 8> w16[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j].p[i] = db[j].p[i] = splat<8>(0.0f);
        if (kKeep && has[j] && !p.w_f32) w16[j] = a.column(p.w, j);
    }
    auto weight = [&](int j) { return !kKeep || p.w_f32 ? a.column(p.w, p.w_f32 != 0, j) : widen<T, 8>(w16[j]); };
    for (int s = 0; s < STAGES; ++s) fetch(first + s * step, mine + uint32_t(s) * STAGE);
    float mu_next[R], rs_next[R];
    auto stats = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = row + r * apart < p.rows;
            mu_next[r] = in ? p.mean[row + r * apart] : 0.0f;
            rs_next[r] = in ? p.rstd[row + r * apart] : 0.0f;
        }
    };
    stats(first);
    uint32_t slot = mine;
    int flip = 0;
    for (int64_t base = base0, row = first; base < p.rows; base += step, row += step, flip ^= 1, xp += x_step) {
        float mu[R], rs[R], sum[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) mu[r] = -mu_next[r], rs[r] = rs_next[r];
        stats(row + step);
        copies_wait<STAGES - 1>();
        int left = 0;  // rows of this thread that exist
#pragma unroll
        for (int r = 0; r < R; ++r) left += row + r * apart < p.rows;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 s1 = splat<8>(0.0f), s2 = s1;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (r >= left || !has[j]) continue;
                const uint32_t at = slot + uint32_t((r * NV + j) * G) * LINE;
                const F32<8> fg = values(at, j), fh = values(at + ARRAY, j), w = weight(j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 gw = mul2(fg.p[i], w.p[i]);
                    s1 = add2(s1, gw);
                    s2 = fma2(gw, add2(fh.p[i], splat<8>(mu[r])), s2);
                }
            }
            sum[2 * r] = total(s1);
            sum[2 * r + 1] = total(s2);
        }
        own_rows_sum<2 * R>(sum, red[flip]);
        // with c = h - mean: dx = (rstd g) w + c (-rstd^2 mean(g u)) + (-rstd mean(g)) + dh, dw = sum (rstd g) c
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 rs2 = splat<8>(rs[r]), c1 = splat<8>(-rs[r] * (sum[2 * r] * p.inv_width)),
                         c2 = splat<8>(-rs[r] * rs[r] * (sum[2 * r + 1] * rs[r] * p.inv_width));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (r >= left || !has[j]) continue;
                const uint32_t at = slot + uint32_t((r * NV + j) * G) * LINE;
                const F32<8> fg = values(at, j), fh = values(at + ARRAY, j), w = weight(j);
                F32<8> v;
                if (has_d) v = values(at + 2 * ARRAY, j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = add2(fh.p[i], splat<8>(mu[r])), t = mul2(fg.p[i], rs2);
                    dw[j].p[i] = fma2(t, c, dw[j].p[i]);
                    db[j].p[i] = add2(fg.p[i], db[j].p[i]);
                    v.p[i] = fma2(c, c2, fma2(t, w.p[i], has_d ? add2(v.p[i], c1) : c1));
                }
                if (G16_CHECK(at_row(xp + r * x_row + j * jump, p.dx, p.lddx, row + r * apart, j)))
                    store_same<T>(reinterpret_cast<T *>(xp + r * x_row + j * jump), v, a.lo(j), a.hi(j));
            }
        }
        fetch(row + STAGES * step, slot);  // this thread has read the slot
        slot += STAGE;
        if (slot == mine + STAGES * STAGE) slot = mine;
    }
    copies_wait<0>();
    if (p.partial == nullptr) return;
    float *out = p.partial + int64_t(blockIdx.x) * 2 * p.width;
    if (kShift || blockDim.y > 1) {
        // through shared memory (the ring holds no copy in flight any more): the block's
        // rows added up in order, and stores that are contiguous over a warp
        float *sums = reinterpret_cast<float *>(ring);
        const int span = int(blockDim.x) * 8 * NV;  // of a row's threads, and behind it as much for dbias
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (kShift || a.at(j) < a.width) {
                    float *to = sums + int(threadIdx.y) * span + a.at(j);
                    if (G16_CHECK(a.at(j) > -8 && a.at(j) + a.o + 8 <= span && smem_window_ok(smem_addr(sums + (int(threadIdx.y) + 1) * span - 1), 4)))
                        store_elems(to, k == 0 ? dw[j] : db[j], a.lo(j), a.hi(j));
                }
            }
            __syncthreads();
            for (int c = tid; c < span && c < a.width; c += int(blockDim.x * blockDim.y)) {
                float s = sums[c];
                for (int y = 1; y < int(blockDim.y); ++y) s += sums[y * span + c];
                if (G16_CHECK(part_ok(p, blockIdx.x, c))) out[k * p.width + c] = s;
            }
        }
        return;
    }
    if constexpr (!kShift) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (a.at(j) >= a.width || !G16_CHECK(part_ok(p, blockIdx.x, a.at(j) + 7))) continue;
            store_f32<float, 8>(out + a.at(j), dw[j]);  // width is a multiple of 8, the workspace aligned
            store_f32<float, 8>(out + p.width + a.at(j), db[j]);
        }
    }
}

// Other rows: longer ones, or off 16-byte boundaries in ways the granules do not take.
// dx with one block per row, which reads its row twice; the column sums by another kernel
// before it, since dx may be written over grad.
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_backward_any_kernel(const LayerNormBackwardArgs p) {
    __shared__ float red[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *g = static_cast<const T *>(p.g) + row * p.ldg, *h = static_cast<const T *>(p.h) + row * p.ldh;
    const T *dh = p.dh != nullptr ? static_cast<const T *>(p.dh) + row * p.lddh : nullptr;
    const float mu = p.mean[row], rs = p.rstd[row];
    auto wg = [&](int64_t at) { return to_f32<T>(g[at]) * load_weight<T, 1>(p.w, p.w_f32 != 0, at).p[0]; };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float v = wg(at);
        s1 += v;
        s2 = fmaf(v, to_f32<T>(h[at]) - mu, s2);
    }
    const float c1 = -rs * (row_sum<false>(s1, red[0]) * p.inv_width), c2 = -rs * (row_sum<false>(s2, red[1]) * rs * p.inv_width);
#pragma unroll 4
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float u = (to_f32<T>(h[at]) - mu) * rs;
        const float v = fmaf(u, c2, fmaf(wg(at), rs, (dh != nullptr ? to_f32<T>(dh[at]) : 0.0f) + c1));
        static_cast<T *>(p.dx)[row * p.lddx + at] = from_f32<T>(v);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const LayerNormBackwardArgs p, int64_t rows_per_block) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t col = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t r0 = int64_t(blockIdx.y) * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < p.rows ? r0 + rows_per_block : p.rows;
    if (col >= p.width) return;
    float dw = 0.0f, db = 0.0f;
#pragma unroll 4
    for (int64_t row = r0; row < r1; ++row) {
        const float g = to_f32<T>(static_cast<const T *>(p.g)[row * p.ldg + col]);
        dw = fmaf(g, (to_f32<T>(static_cast<const T *>(p.h)[row * p.ldh + col]) - p.mean[row]) * p.rstd[row], dw);
        db += g;
    }
    float *out = p.partial + int64_t(blockIdx.y) * 2 * p.width + col;
    if (!G16_CHECK(part_ok(p, blockIdx.y, col))) return;
    out[0] = dw;
    out[p.width] = db;
}

// The parts' sums of dweight and dbias: 32 columns per block, blockDim.y threads each add
// every blockDim.y-th part, then the first adds theirs in order. Either may be absent.
constexpr int kPartThreads = 32;
__global__ void __launch_bounds__(32 * kPartThreads) sum_parts_kernel(const float *partial, float *dweight, float *dbias,
                                                                      int64_t parts, int64_t width) {
    __shared__ float s[kPartThreads][33];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;  // of both gradients, one behind the other
    float *out = col < width ? dweight : dbias;
    const bool live = col < 2 * width && out != nullptr;
    float v = 0.0f;
    if (live) {
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < parts; r += kPartThreads) v += __ldcg(partial + r * 2 * width + col);
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || !live) return;
    for (int g = 1; g < kPartThreads; ++g) v += s[g][threadIdx.x];
    out[col < width ? col : col - width] = v;
}

// ------------------------------------------------------------------ launch shapes
struct RowShape {
    int nv;        // loads of 8 elements per thread
    int tpr, rpb;  // threads per row, rows per block
    bool fits;     // the row fits its threads' registers
};

// One load per thread where 1024 threads hold the row so, else the fewest, but not fewer
// than `least`; short rows share a block of 256 threads.
RowShape row_shape(int64_t width, int least) {
    RowShape s{1, 32, 1, false};
    for (int nv : {1, 2, 4}) {
        const int64_t t = cdiv(cdiv(width, 8 * nv), 32) * 32;
        if (t > 1024 || nv < least) continue;
        s.nv = nv;
        s.tpr = int(t);
        s.fits = true;
        break;
    }
    if (s.fits && s.tpr <= 128) s.rpb = 256 / s.tpr;
    return s;
}

// Shared memory of the forms that keep a row's values: 0 where they do not fit.
constexpr int kKeptBytes = 200 * 1024;
int kept_bytes(int64_t width) { return width * 4 <= kKeptBytes ? int(width * 4) : 0; }
int any_threads(int64_t width) { return int(std::min<int64_t>(1024, std::max<int64_t>(32, cdiv(cdiv(width, 4), 32) * 32))); }

// One load per thread for up to two rows an SM, where the chain load - sums - store is
// what counts; then more, so that blocks are small and several on an SM are at different
// points of it: two (1000 x 4096 bf16 with residual, one / two / four loads: 10.3 / 7.8 /
// 8.1 us, 2000 x 4096 17.9 / 13.0 / 14.4, 8192 x 4096 63.8 / 44.2 / 44.2), four of long rows
// (4096 x 8192 72.9 / 47.2 / 44.3, to 8 bits 76.7 / 48.2 / 40.9). fp32's are twice as long
// (4096 x 4096 49.9 / 53.2 / 55.8).
int norm_loads(int64_t rows, int64_t width, size_t es, int num_sms) {
    if (es == 4 || rows <= 2 * num_sms) return 1;
    return width < 8192 ? 2 : 4;
}
// Of two and four loads the one whose blocks leave fewer of an SM's threads idle (64
// registers each), where that counts: 8191 elements take 544 threads with two loads, one
// block on an SM, 288 with four, three (4096 x 8191 87 us with two).
RowShape norm_shape(int64_t rows, int64_t width, size_t es, int num_sms) {
    const int least = norm_loads(rows, width, es, num_sms);
    const RowShape s = row_shape(width, least), t = row_shape(width, 4);
    auto busy = [](const RowShape &r) { return r.tpr > 0 ? 1024 / (r.tpr * r.rpb) * (r.tpr * r.rpb) : 0; };
    return least == 2 && s.fits && t.fits && busy(s) * 100 < busy(t) * 85 ? t : s;
}
// Without weights and further sums, four (16384 x 1024 bf16 11.5 / 9.8 / 9.1 us, 4096 x 16384
// 38.3 / 38.0 / 32.7, 300 x 4096 1.5 / 1.7 / 1.7).
int quantize_loads(int64_t rows, size_t es, int num_sms) { return es == 4 || rows <= 2 * num_sms ? 1 : 4; }

template <typename T, int OUT>
cudaError_t norm(const LayerNormArgs &p, int num_sms, cudaStream_t stream) {
    auto go = [&](auto *k, const RowShape &s) {
        return launch(k, dim3(unsigned(cdiv(p.rows, s.rpb))), dim3(unsigned(s.tpr), unsigned(s.rpb)), 0, stream, p);
    };
    if constexpr (sizeof(T) == 2) {
        const RowShape s = norm_shape(p.rows, p.width + 7, sizeof(T), num_sms);
        if (p.shift && s.fits)
            return go(s.nv == 1   ? layer_norm_kernel<T, 1, OUT, true>
                      : s.nv == 2 ? layer_norm_kernel<T, 2, OUT, true>
                                  : layer_norm_kernel<T, 4, OUT, true>, s);
    }
    const RowShape s = norm_shape(p.rows, p.width, sizeof(T), num_sms);
    if (p.vec && s.fits)
        return go(s.nv == 1   ? layer_norm_kernel<T, 1, OUT, false>
                  : s.nv == 2 ? layer_norm_kernel<T, 2, OUT, false>
                              : layer_norm_kernel<T, 4, OUT, false>, s);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = allow_smem<layer_norm_any_kernel<T, OUT>>(dev, kKeptBytes);
    if (e != cudaSuccess) return e;
    const int kept = kept_bytes(p.width);
    return launch(layer_norm_any_kernel<T, OUT>, dim3(unsigned(p.rows)), dim3(unsigned(any_threads(p.width))), kept, stream, p,
                  int32_t(kept > 0));
}

template <typename T, int OUT>
cudaError_t quantize(const QuantizeArgs &p, int num_sms, cudaStream_t stream) {
    const int least = quantize_loads(p.rows, sizeof(T), num_sms);
    auto go = [&](auto *k, const RowShape &s) {
        return launch(k, dim3(unsigned(cdiv(p.rows, s.rpb))), dim3(unsigned(s.tpr), unsigned(s.rpb)), 0, stream, p);
    };
    if constexpr (sizeof(T) == 2) {
        const RowShape s = row_shape(p.width + 7, least);
        if (p.shift && s.fits)
            return go(s.nv == 1   ? quantize_rows_kernel<T, 1, OUT, true>
                      : s.nv == 2 ? quantize_rows_kernel<T, 2, OUT, true>
                                  : quantize_rows_kernel<T, 4, OUT, true>, s);
    }
    const RowShape s = row_shape(p.width, least);
    if (p.vec && s.fits)
        return go(s.nv == 1   ? quantize_rows_kernel<T, 1, OUT, false>
                  : s.nv == 2 ? quantize_rows_kernel<T, 2, OUT, false>
                              : quantize_rows_kernel<T, 4, OUT, false>, s);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = allow_smem<quantize_any_kernel<T, OUT>>(dev, kKeptBytes);
    if (e != cudaSuccess) return e;
    const int kept = kept_bytes(p.width);
    return launch(quantize_any_kernel<T, OUT>, dim3(unsigned(p.rows)), dim3(unsigned(any_threads(p.width))), kept, stream, p,
                  int32_t(kept > 0));
}

// The persistent backward form: one block of up to 512 threads (128 registers each) on an
// SM, NV loads of 8 elements per thread and as many rows side by side as there are threads
// for; NV by how many of the threads' loads are used. A step's copies take 16 bytes of each
// array for every load of a thread (32 of fp32).
struct BackwardPlan {
    bool ok, shift;
    int nv, rpt, tpr, rpb, grid;
};

template <typename T>
BackwardPlan plan_backward(const LayerNormBackwardArgs &p, int num_sms) {
    BackwardPlan b{};
    b.shift = sizeof(T) == 2 && p.shift;
    if (!p.vec && !b.shift) return b;
    const int64_t loads = cdiv(p.width + (b.shift ? 7 : 0), 8);
    // one load per thread for few rows, whose chain is then short, and for short ones (64 x
    // 4096 6.1 / 8.2 us with two, 300 x 4096 8.6 / 10.3, 4096 x 768 12.3 / 13.2); else two (8192 x
    // 4096 56.2 / 50.7, with three 56.4), more where the row needs them
    b.nv = loads <= 512 && (p.rows <= 2 * num_sms || loads <= 128) ? 1 : loads <= 1024 ? 2 : loads <= 1536 ? 3 : 4;
    if (loads > (sizeof(T) == 2 ? 2048 : 1024)) return b;
    b.tpr = int(cdiv(cdiv(loads, b.nv), 32) * 32);
    if (b.tpr > kBackThreads) return b;
    b.rpb = std::min(kBackThreads / b.tpr, 15);  // a barrier each, besides the block's
    // shifted: a thread's rows are 8 k apart, or it has one row only
    const bool one_row = b.shift && cdiv(p.rows, b.rpb) <= num_sms;
    b.rpt = sizeof(T) == 4 || b.nv > 2 || one_row ? 1 : 2;
    // as few blocks, and parts of the column sums, as take the same number of steps
    const int64_t units = cdiv(p.rows, b.rpb * b.rpt);
    b.grid = int(cdiv(units, cdiv(units, num_sms)));
    if (b.shift && !one_row) {
        if (num_sms < 8) return b;
        b.grid = int(std::min<int64_t>(cdiv(b.grid, 8) * 8, num_sms / 8 * 8));
    }
    b.ok = true;
    return b;
}

template <typename T, int NV, int R, int STAGES, bool kShift>
cudaError_t backward_rows(const LayerNormBackwardArgs &p, const BackwardPlan &b, int dev, cudaStream_t stream) {
    constexpr int per_thread = 16 * (int(sizeof(Raw<T, 8>)) / 16) * 3 * NV * R * STAGES, sums = NV * 8 * 4;
    static_assert(per_thread >= sums, "the sums' way out fits the ring");
    static_assert(kBackThreads * per_thread + 4 * R * 32 * 4 <= 226 * 1024, "shared memory of an SM");
    const cudaError_t e = allow_smem<layer_norm_backward_rows_kernel<T, NV, R, STAGES, kShift>>(dev, kBackThreads * per_thread);
    if (e != cudaSuccess) return e;
    return launch(layer_norm_backward_rows_kernel<T, NV, R, STAGES, kShift>, dim3(unsigned(b.grid)),
                  dim3(unsigned(b.tpr), unsigned(b.rpb)), kBackThreads * per_thread, stream, p);
}

template <typename T, bool kShift>
cudaError_t backward_rows(const LayerNormBackwardArgs &p, const BackwardPlan &b, int dev, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) {
        return b.nv == 1 ? backward_rows<T, 1, 1, 4, kShift>(p, b, dev, stream) : backward_rows<T, 2, 1, 2, kShift>(p, b, dev, stream);
    } else {
        if (b.nv == 1)
            return b.rpt == 1 ? backward_rows<T, 1, 1, 4, kShift>(p, b, dev, stream) : backward_rows<T, 1, 2, 4, kShift>(p, b, dev, stream);
        if (b.nv == 2)
            return b.rpt == 1 ? backward_rows<T, 2, 1, 4, kShift>(p, b, dev, stream) : backward_rows<T, 2, 2, 2, kShift>(p, b, dev, stream);
        return b.nv == 3 ? backward_rows<T, 3, 1, 3, kShift>(p, b, dev, stream) : backward_rows<T, 4, 1, 2, kShift>(p, b, dev, stream);
    }
}

template <typename T>
cudaError_t backward(const LayerNormBackwardArgs &p, float *dweight, float *dbias, int dev, int num_sms, cudaStream_t stream) {
    const BackwardPlan b = plan_backward<T>(p, num_sms);
    cudaError_t e = cudaSuccess;
    int64_t parts;
    if (b.ok) {
        parts = b.grid;
        if (!b.shift) e = backward_rows<T, false>(p, b, dev, stream);
        else if constexpr (sizeof(T) == 2) e = backward_rows<T, true>(p, b, dev, stream);
    } else {
        const int64_t rows_per_block = cdiv(p.rows, kLayerNormParts);
        parts = cdiv(p.rows, rows_per_block);
        if (p.partial != nullptr)
            e = launch(layer_norm_columns_kernel<T>, dim3(unsigned(cdiv(p.width, 256)), unsigned(parts)), dim3(256), 0, stream, p,
                       rows_per_block);
        if (e == cudaSuccess)
            e = launch(layer_norm_backward_any_kernel<T>, dim3(unsigned(p.rows)), dim3(unsigned(any_threads(p.width))), 0, stream, p);
    }
    if (e == cudaSuccess && p.partial != nullptr)
        e = launch(sum_parts_kernel, dim3(unsigned(cdiv(2 * p.width, 32))), dim3(32, kPartThreads), 0, stream,
                   static_cast<const float *>(p.partial), dweight, dbias, parts, p.width);
    return e;
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs &p, int num_sms, cudaStream_t stream) {
    auto typed = [&](auto zero) {
        using T = decltype(zero);
        if (p.out == kOutE4m3) return norm<T, kOutE4m3>(p, num_sms, stream);
        if (p.out == kOutI8) return norm<T, kOutI8>(p, num_sms, stream);
        return norm<T, kOutSame>(p, num_sms, stream);
    };
    return p.type == 0 ? typed(float()) : p.type == 1 ? typed(__half()) : typed(__nv_bfloat16());
}

cudaError_t launch_layer_norm_backward(const LayerNormBackwardArgs &p, float *dweight, float *dbias, int dev, int num_sms,
                                       cudaStream_t stream) {
    if (p.type == 0) return backward<float>(p, dweight, dbias, dev, num_sms, stream);
    if (p.type == 1) return backward<__half>(p, dweight, dbias, dev, num_sms, stream);
    return backward<__nv_bfloat16>(p, dweight, dbias, dev, num_sms, stream);
}

cudaError_t launch_quantize_rows(const QuantizeArgs &p, int num_sms, cudaStream_t stream) {
    auto typed = [&](auto zero) {
        using T = decltype(zero);
        return p.out == kOutI8 ? quantize<T, kOutI8>(p, num_sms, stream) : quantize<T, kOutE4m3>(p, num_sms, stream);
    };
    return p.type == 0 ? typed(float()) : p.type == 1 ? typed(__half()) : typed(__nv_bfloat16());
}

}  // namespace g16
