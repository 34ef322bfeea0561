// 8-bit rows in front of 16-bit products (sm_103a): whole numbers and 8-bit floats to
// 16 bits, and the elementwise part of a product's backward pass from 8-bit values.
//
// A whole number of 8 bits is exact in fp16, and so is the product of two in the fp32
// sums of the 16-bit tensor cores (11-bit factors); a sum is exact to 2^24 and from
// there on rounded like any other fp32 sum. sm_103a's tensor cores have no integer kind at
// a rate worth using, and 8-bit floats hold no whole numbers past 16.
#pragma once
#include "ops_linear.cuh"

namespace g16 {

constexpr uint32_t kEightE4m3 = 3, kEightI8 = 4;  // GEMM_TYPE_*

// Four whole numbers of 8 bits -> fp16, exactly: with the sign bit turned x is x + 128 in
// 0 .. 255; 0x6400 | that is 1024 + 128 + x in fp16.
__device__ __forceinline__ uint2 i8x4_to_f16(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x5140), b = __byte_perm(u, 0x64646464u, 0x7362);
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias), hb = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&ha), *reinterpret_cast<const uint32_t *>(&hb));
}

// Eight 8-bit elements as their values.
__device__ __forceinline__ F32<8> eight_values(uint2 w, uint32_t type) {
    uint2 lo, hi;  // fp16
    if (type == kEightI8) {
        lo = i8x4_to_f16(w.x);
        hi = i8x4_to_f16(w.y);
    } else {
        auto pair = [](uint32_t v) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(v), __NV_E4M3);
            return uint32_t(h.x) | (uint32_t(h.y) << 16);
        };
        lo = make_uint2(pair(w.x & 0xffffu), pair(w.x >> 16));
        hi = make_uint2(pair(w.y & 0xffffu), pair(w.y >> 16));
    }
    F32<8> v;
    v.p[0] = unpack2<__half>(lo.x);
    v.p[1] = unpack2<__half>(lo.y);
    v.p[2] = unpack2<__half>(hi.x);
    v.p[3] = unpack2<__half>(hi.y);
    return v;
}

// Bytes 0 .. 7 from p on, of which n are the row's (n >= 1; the others are not to be
// used), past L1. From the one or two aligned words that hold the row's bytes.
template <bool kAligned>
__device__ __forceinline__ uint2 load_eight(const uint8_t *p, int64_t n) {
    if constexpr (kAligned) return __ldcg(reinterpret_cast<const uint2 *>(p));
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t s = uint32_t(at & 7u);
    const uint2 *w = reinterpret_cast<const uint2 *>(at - s);
    const uint2 a = __ldcg(w);
    if (s == 0) return a;
    uint2 b = make_uint2(0u, 0u);
    if (int64_t(s) + (n < 8 ? n : 8) > 8) b = __ldcg(w + 1);
    const uint32_t v[4] = {a.x, a.y, b.x, b.y};
    const uint32_t k = s >> 2, bits = (s & 3u) * 8u;
    const uint32_t x = k ? v[1] : v[0], y = k ? v[2] : v[1], z = k ? v[3] : v[2];
    return make_uint2(__funnelshift_r(x, y, bits), __funnelshift_r(y, z, bits));
}

// ------------------------------------------------------------------ 8 bits -> 16
// Rows of `inner` 8-bit elements, any base and pitch -> rows of 16-bit ones on 128-byte
// lines (dst 128-byte aligned, ld_dst a multiple of 64), zero in the rest of a row's last
// granule. kPlain: whole numbers as they are, in fp16. Else act(scale x), rounded to T.
// A thread has one granule of the copy in every row it visits, four rows at a time. Bound by
// DRAM, one byte read and two written.
struct ExpandJob {
    const uint8_t *src;
    void *dst;
    const float *scale;  // of each row; not kPlain
    int64_t rows, inner, ld_src, ld_dst;
    uint32_t type, act;  // of the source; not kPlain
    int32_t lg;          // 2^lg granules of a row, 256 >> lg rows per block and step
    int32_t bx, by;      // blocks along a row, along the rows; 0: no job
};

template <typename T, bool kPlain, bool kAligned, uint32_t ACT>
__device__ __forceinline__ void expand_rows(const ExpandJob &J, int block) {
    const int tx = int(threadIdx.x) & ((1 << J.lg) - 1), ty = int(threadIdx.x) >> J.lg, per = 256 >> J.lg;
    const int64_t i0 = 8 * ((int64_t(block % J.bx) << J.lg) + tx);
    if (i0 >= J.inner) return;
    const int64_t left = J.inner - i0, step = int64_t(J.by) * per;
    constexpr int AHEAD = 4;
#pragma unroll 1
    for (int64_t r = int64_t(block / J.bx) * per + ty; r < J.rows; r += AHEAD * step) {
        uint2 w[AHEAD];
        float s[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * step;
            if (row >= J.rows) break;
            w[k] = load_eight<kAligned>(J.src + row * J.ld_src + i0, left);
            if constexpr (!kPlain) s[k] = __ldcg(J.scale + row);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * step;
            if (row >= J.rows) break;
            if (!G16_CHECK(i0 + 8 <= J.ld_dst)) continue;
            Raw<T, 8> out;
            if constexpr (kPlain) {
                const uint2 lo = i8x4_to_f16(w[k].x), hi = i8x4_to_f16(w[k].y);
                out.q[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                F32<8> v = eight_values(w[k], J.type);
#pragma unroll
                for (int i = 0; i < 4; ++i) v.p[i] = act_value<ACT>(mul2(v.p[i], pair_of(s[k])));
                out.q[0] = make_uint4(pack2<T>(v.p[0]), pack2<T>(v.p[1]), pack2<T>(v.p[2]), pack2<T>(v.p[3]));
            }
            if (left < 8) keep_elems<T>(out, 0, int(left));
            *reinterpret_cast<uint4 *>(static_cast<T *>(J.dst) + row * J.ld_dst + i0) = out.q[0];
        }
    }
}

template <typename T, bool kPlain>
__global__ void __launch_bounds__(256) expand_rows_kernel(const ExpandJob a, const ExpandJob b) {
    griddep_wait();
    griddep_launch_dependents();
    const bool second = int(blockIdx.x) >= a.bx * a.by;
    const ExpandJob &J = second ? b : a;
    const int block = int(blockIdx.x) - (second ? a.bx * a.by : 0);
    const bool aligned = ((reinterpret_cast<uintptr_t>(J.src) | uintptr_t(J.ld_src)) & 7u) == 0;
    if constexpr (kPlain) {
        if (aligned) expand_rows<T, true, true, kActNone>(J, block);
        else expand_rows<T, true, false, kActNone>(J, block);
    } else {
        auto run = [&](auto act) {
            constexpr uint32_t ACT = decltype(act)::value;
            if (aligned) expand_rows<T, false, true, ACT>(J, block);
            else expand_rows<T, false, false, ACT>(J, block);
        };
        switch (J.act) {
            case kActRelu: run(std::integral_constant<uint32_t, kActRelu>()); break;
            case kActGelu: run(std::integral_constant<uint32_t, kActGelu>()); break;
            case kActGeluTanh: run(std::integral_constant<uint32_t, kActGeluTanh>()); break;
            case kActSilu: run(std::integral_constant<uint32_t, kActSilu>()); break;
            default: run(std::integral_constant<uint32_t, kActNone>()); break;
        }
    }
}

// ------------------------------------------------------------------ D from 8-bit values
// D = G act'(s P8) and the column sums of D over blocks of rows: linear_grad_kernel with
// the values before the activation in 8 bits and a scale per row.
struct SavedGradParams {
    GradParams g;  // pre: the 8-bit values, ldp their pitch
    const float *scale;
    uint32_t type;
};

template <uint32_t ACT, typename T, bool kShift>
__device__ __forceinline__ void saved_grad_rows(const SavedGradParams &s, int64_t col, int64_t r0, int64_t r1, F32<8> &sum) {
    const GradParams &p = s.g;
    const T *g = static_cast<const T *>(p.g);
    const uint8_t *pre = static_cast<const uint8_t *>(p.pre);
    T *d = static_cast<T *>(p.d);
    constexpr int AHEAD = kShift ? 2 : 4;  // rows loaded before the first is stored
#pragma unroll 1
    for (int64_t r = r0 + threadIdx.y; r < r1; r += AHEAD * kGradGroups) {
        GradLoad<T, kShift> a[AHEAD];
        uint2 b[AHEAD];
        float f[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * kGradGroups;
            if (row >= r1) break;
            a[k].fetch(g + row * p.ldg, col, p.N);
            b[k] = load_eight<!kShift>(pre + row * p.ldp + col, p.N - col);
            f[k] = __ldcg(s.scale + row);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * kGradGroups;
            if (row >= r1) break;
            F32<8> x = a[k].values(g + row * p.ldg, col, p.N);
            const F32<8> v = eight_values(b[k], s.type);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.p[i] = mul2(x.p[i], act_slope<ACT>(mul2(v.p[i], pair_of(f[k]))));
            if (kShift && col + 8 > p.N) {  // columns past the last hold another's bytes
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (col + 2 * i >= p.N) x.p[i].x = 0.0f;
                    if (col + 2 * i + 1 >= p.N) x.p[i].y = 0.0f;
                }
            }
            if (d != nullptr) {
                if constexpr (kShift) store_some<T>(d + row * p.ldd + col, x, 0, int(p.N - col < 8 ? p.N - col : 8));
                else store_f32<T, 8>(d + row * p.ldd + col, x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum.p[i] = add2(sum.p[i], x.p[i]);
        }
    }
}

// kShift: G's rows off 16-byte or pre's off 8-byte boundaries, or N no multiple of 8.
template <typename T, bool kShift>
__global__ void __launch_bounds__(32 * kGradGroups) saved_grad_kernel(const SavedGradParams s) {
    __shared__ float part[kGradGroups][32 * 8 + 1];
    const GradParams &p = s.g;
    griddep_enter(p.late);
    const int64_t col = (int64_t(blockIdx.x) * 32 + threadIdx.x) * 8;
    const int64_t r0 = int64_t(blockIdx.y) * p.rows_per_block;
    const int64_t r1 = r0 + p.rows_per_block < p.M ? r0 + p.rows_per_block : p.M;
    F32<8> sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum.p[i] = pair_of(0.0f);
    if (col < p.N) {
        switch (p.act) {
            case kActRelu: saved_grad_rows<kActRelu, T, kShift>(s, col, r0, r1, sum); break;
            case kActGelu: saved_grad_rows<kActGelu, T, kShift>(s, col, r0, r1, sum); break;
            case kActGeluTanh: saved_grad_rows<kActGeluTanh, T, kShift>(s, col, r0, r1, sum); break;
            default: saved_grad_rows<kActSilu, T, kShift>(s, col, r0, r1, sum); break;
        }
    }
    griddep_leave(p.late);
    if (p.partial == nullptr) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        part[threadIdx.y][threadIdx.x * 8 + 2 * i] = sum.p[i].x;
        part[threadIdx.y][threadIdx.x * 8 + 2 * i + 1] = sum.p[i].y;
    }
    __syncthreads();
    for (int c = threadIdx.y * 32 + threadIdx.x; c < 32 * 8; c += 32 * kGradGroups) {
        const int64_t at = int64_t(blockIdx.x) * 32 * 8 + c;
        if (at >= p.N) continue;
        float v = part[0][c];
        for (int y = 1; y < kGradGroups; ++y) v += part[y][c];
        p.partial[int64_t(blockIdx.y) * p.N + at] = v;
    }
}

}  // namespace g16
