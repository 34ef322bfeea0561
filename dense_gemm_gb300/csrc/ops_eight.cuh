// 8-bit rows in front of 16-bit products (sm_103a): whole numbers and 8-bit floats to
// 16 bits, and the elementwise part of a product's backward pass from 8-bit values.
//
// A whole number of 8 bits is exact in fp16, and so is the product of two in the fp32
// sums of the 16-bit tensor cores (11-bit factors); a sum is exact while that of the
// magnitudes is below 2^24, and from there on an addition may lose 2^-23 of them. sm_103a's tensor cores have no integer kind at
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
// granule. (A 16-bit source: copy_rows.) kPlain: whole numbers as they are, in fp16. Else act(scale x), rounded to T.
// A thread has one granule of the copy in every row it visits, eight rows at a time. Bound by
// DRAM, one byte read and two written, and with an activation by its arithmetic. (Two
// granules per thread: stores 32 bytes apart, 27 million whole numbers 17.9 us instead of 12.0.)
struct ExpandJob {
    const uint8_t *src;
    void *dst;
    const float *scale;  // of each row; not kPlain
    int64_t rows, inner, ld_src, ld_dst;
    uint32_t type, act;  // of the source; not kPlain
    int32_t lg;          // 2^lg granules of a row, 256 >> lg rows per block and step
    int32_t bx, by;      // blocks along a row, along the rows; 0: no job
};
constexpr int kExpandAhead = 8;

template <typename T, bool kPlain, bool kAligned, uint32_t ACT>
__device__ __forceinline__ void expand_rows(const ExpandJob &J, int block) {
    const int tx = int(threadIdx.x) & ((1 << J.lg) - 1), ty = int(threadIdx.x) >> J.lg, per = 256 >> J.lg;
    const int64_t i0 = 8 * ((int64_t(block % J.bx) << J.lg) + tx);
    if (i0 >= J.inner) return;
    const int64_t left = J.inner - i0, step = int64_t(J.by) * per;
    constexpr int AHEAD = kAligned ? kExpandAhead : kExpandAhead / 2;
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

// Rows of 16-bit elements off 16-byte boundaries onto 128-byte lines, in the same launch: a
// granule of the copy from the one or two that hold its elements (257 x 1000 x 513: a
// launch less, 19.4 -> 18.5 us of device time).
template <typename T>
__device__ __forceinline__ void copy_rows(const ExpandJob &J, int block) {
    const int tx = int(threadIdx.x) & ((1 << J.lg) - 1), ty = int(threadIdx.x) >> J.lg, per = 256 >> J.lg;
    const int64_t i0 = 8 * ((int64_t(block % J.bx) << J.lg) + tx);
    if (i0 >= J.inner) return;
    const int64_t left = J.inner - i0, step = int64_t(J.by) * per;
    constexpr int AHEAD = kExpandAhead / 2;
#pragma unroll 1
    for (int64_t r = int64_t(block / J.bx) * per + ty; r < J.rows; r += AHEAD * step) {
        GradLoad<T, true> v[AHEAD];
        const T *src = reinterpret_cast<const T *>(J.src);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (r + k * step < J.rows) v[k].fetch(src + (r + k * step) * J.ld_src, i0, J.inner);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * step;
            if (row >= J.rows || !G16_CHECK(i0 + 8 <= J.ld_dst)) break;
            Raw<T, 8> out = shift_granules<T>(v[k].lo, v[k].hi, place_in_granule(src + row * J.ld_src + i0));
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
    if constexpr (!kPlain) {
        if (J.type < kEightE4m3) {
            copy_rows<T>(J, block);
            return;
        }
    }
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

// ================================================================== linear_int8
// Few rows of C, 8-bit integers: linear_split's tiles and sums with the weights' stream in 8
// bits. A stage is 128 weights' rows and T tokens by 128 bytes of K. It lands by TMA as it
// is; four of eight warps turn it into fp16, each thread a row: the weights from registers into
// tensor memory, where the MMA takes its 128-row operand from, the tokens into shared memory.
// kWide, more than 64 tokens: converting them in every CTA would take longer than the weights,
// so they come as fp16 (a kernel before this one made a copy of them) in a ring of their own.
// (As fp16 in shared memory the weights would be written once and read once more there: 32
// KiB each way a stage, beside the 16 in and 16 out of their bytes, on an SM that gets 16 KiB
// of weights in 0.36 us from DRAM and moves 128 bytes a cycle.)
namespace lin {
constexpr int I8_W_BYTES = SPLIT_ROWS * 128;  // weights of a stage
constexpr int I8_COPIES = 2;                  // stages in fp16, one of each group of warps
constexpr int I8_MAX_STAGES = 6, I8_MAX_X = 4;
constexpr int I8_A_COLS = 64;                 // TMEM columns of a stage's weights: 128 of K, two to a column
// full[S], empty[S], ready[2], used[2], done, kWide's tokens: full[4], empty[4]
constexpr int I8_BARS = 2 * I8_MAX_STAGES + 2 * I8_COPIES + 1 + 2 * I8_MAX_X;
// stages of weights, and of tokens: in 8 bits beside the weights with two copies in fp16, or (wide) x stages in fp16
constexpr int i8_ring(bool wide, int stages, int x, int T) {
    return stages * I8_W_BYTES + (wide ? x * T * 256 : stages * T * 128 + I8_COPIES * T * 256);
}
constexpr int i8_smem(bool wide, int stages, int x, int T) { return i8_ring(wide, stages, x, T) + I8_BARS * 8 + 16 + 1024; }
}  // namespace lin

// 32 lanes x 32 consecutive 32-bit columns from registers: thread i has lane (base lane + i).
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    if (!__all_sync(0xffffffffu, G16_CHECK((taddr & 0xFFFFu) + 32u <= 512u))) return;
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc], fp16 x fp16 -> fp32: A's rows are the lanes, two
// elements of K to a column.
__device__ __forceinline__ void mma_f16_tmem_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred pe, pa;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "setp.ne.b32 pa, %4, 0;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pa;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Cluster of p.split CTAs along x, all on the same tile of 128 columns by T rows of C; CTA
// r sums the stages r n / split ... (r + 1) n / split of n.
// Bound by the weights' stream where N K is large and rows are few (1 x 16384 x 4096 67 MB in
// 15.8 us, floor 9.9), else by the chain set-up - first weights - conversion - exchange - rows (1 x
// 4096 x 4096 7.4 us of which the stream is 2.5) and from 32 rows on by the conversion: a stage takes a
// group some 1400 cycles with 16 tokens, 2700 with 64 (64 x 16384 x 4096 19.8 us). kWide with T = 256 by
// shared memory's bandwidth: 0.86 us a stage, 16 KiB of weights in and out and 64 of tokens, for
// 0.54 of products (256 x 8192 x 8192 33.1 us, 512 57, 256 x 4096 x 4096 17.0).
template <bool kWide>
__global__ void __launch_bounds__(lin::SPLIT_THREADS, 2)
    linear_int8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinearParams p) {
    constexpr int MMA_WARP = 1, EPI_WARP0 = 2;
    const int NST = p.stages, T = p.T;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // same offset in every CTA of the cluster
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t x_bytes = uint32_t(T) * 128u;
    const uint32_t sW = base, sX = base + uint32_t(NST) * lin::I8_W_BYTES;
    const uint32_t sX16 = kWide ? sX : sX + uint32_t(NST) * x_bytes;
    const int XST = kWide ? p.bufs : lin::I8_COPIES;  // stages of tokens in fp16
    const uint32_t ring = sX16 + uint32_t(XST) * 2u * x_bytes - base;
    const uint32_t bar0 = base + ring;
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (lin::I8_MAX_STAGES + s); };
    auto ready_bar = [&](uint32_t s) { return bar0 + 8u * (2 * lin::I8_MAX_STAGES + s); };
    auto used_bar = [&](uint32_t s) { return bar0 + 8u * (2 * lin::I8_MAX_STAGES + lin::I8_COPIES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * lin::I8_MAX_STAGES + 2 * lin::I8_COPIES);
    auto x_full = [&](uint32_t s) { return done_bar + 8u * (1u + s); };
    auto x_empty = [&](uint32_t s) { return done_bar + 8u * (1u + lin::I8_MAX_X + s); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + ring + lin::I8_BARS * 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int S = p.split;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    // rows of C vary fastest, so that the CTAs sharing weights run together
    const int32_t tile = int32_t(blockIdx.x) / S;
    const int32_t tn = tile / p.sched.nm, tm = tile - tn * p.sched.nm;
    const int32_t m0 = tm * T, n0 = tn * lin::SPLIT_ROWS;
    const int32_t steps = p.num_kb;  // stages of the whole sum
    const int32_t st0 = int32_t(int64_t(steps) * rank / S), st1 = int32_t(int64_t(steps) * (rank + 1) / S);
    const int valid = int(p.M - m0 < T ? p.M - m0 : T);  // rows of C in this tile
    const int acc_cols = T < 32 ? 32 : T;                // the weights' stages follow the accumulator

    bool ready = false;  // epilogue warps: the accumulator is complete
    uint32_t tmem_base = 0;
    const int ew = warp - EPI_WARP0;
    const bool vec = p.e.vec4 && int64_t(n0) + lin::SPLIT_ROWS <= p.N;  // n0 may lie within 128 of 2^31
    SplitColumns columns = {};

    auto load = [&](int32_t st, uint32_t stage) {
        mbar_expect_tx_elect(full_bar(stage), kWide ? lin::I8_W_BYTES : lin::I8_W_BYTES + x_bytes);
        tma_load_2d_elect<false>(sW + stage * lin::I8_W_BYTES, &tmW, st * 128, n0, full_bar(stage));
        if constexpr (!kWide) tma_load_2d_elect<false>(sX + stage * x_bytes, &tmX, st * 128, m0, full_bar(stage));
    };
    // kWide: both k-blocks of 64 of the tokens
    auto load_x = [&](auto mode, int32_t st, uint32_t stage) {
        mbar_expect_tx_elect(x_full(stage), 2u * x_bytes);
        issue_copies<decltype(mode)::value, false, false>(&tmX, sX16 + stage * 2u * x_bytes, x_bytes, p.a.copies, 2 * st, 64, m0,
                                                          x_full(stage), lane);
    };
    if (warp == 0) {
        // ============================================================ producer
        if (lane == 0) {
            prefetch_tensormap(&tmW);
            prefetch_tensormap(&tmX);
            for (int s = 0; s < NST; ++s) {
                mbar_init(full_bar(s), 1);
                mbar_init(empty_bar(s), EPI_WARPS / 2);
            }
            for (int s = 0; s < lin::I8_COPIES; ++s) {
                mbar_init(ready_bar(s), EPI_WARPS / 2);
                mbar_init(used_bar(s), 1);
            }
            mbar_init(done_bar, 1);
            for (int s = 0; kWide && s < XST; ++s) {
                mbar_init(x_full(s), 1);
                mbar_init(x_empty(s), 1);
            }
            fence_mbar_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
        const int32_t first = min(st0 + NST, st1);
        // the first stages' weights are on their way into L2 while the kernel before ends
        for (int32_t st = st0; st < first; ++st) prefetch_copies<kLoadOne, false>(&tmW, st, 128, n0);
        // kWide: the kernel before is the tokens' copy, which the weights need nothing of: what they
        // hold was complete before that kernel's own wait returned, and so before this one could start
        if constexpr (!kWide) griddep_wait();
        for (int32_t st = st0; st < first; ++st) load(st, uint32_t(st - st0));
        auto later_stages = [&](auto mode) {
            __syncthreads();  // the others are set up; tensor memory is allocated
            if constexpr (kWide) {
                griddep_wait();
                for (int32_t st = st0; st < min(st0 + XST, st1); ++st) load_x(mode, st, uint32_t(st - st0));
            }
            griddep_launch_dependents();
            // kWide: the tokens' ring may be shorter than the weights', which then are as many stages ahead
            uint32_t stage = 0, phase = 0;
            [[maybe_unused]] uint32_t x_stage = 0, x_phase = 0;
            for (int32_t st = st0 + (kWide ? XST : NST); st < st1; ++st) {
                const int32_t ws = kWide ? st + NST - XST : st;
                if (ws < st1) {
                    if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase, p.wait))) {
                        let_copies_land();
                        break;
                    }
                    load(ws, stage);
                    if (++stage == uint32_t(NST)) { stage = 0; phase ^= 1u; }
                }
                if constexpr (kWide) {
                    if (!__all_sync(0xffffffffu, mbar_wait(x_empty(x_stage), x_phase, p.wait))) {
                        let_copies_land();
                        break;
                    }
                    load_x(mode, st, x_stage);
                    if (++x_stage == uint32_t(XST)) { x_stage = 0; x_phase ^= 1u; }
                }
            }
            __syncwarp();
        };
        if constexpr (kWide) with_load(p.a, [&](auto mode, auto) { later_stages(mode); });
        else later_stages(std::integral_constant<uint32_t, kLoadOne>());
    } else {
        if (warp == MMA_WARP) {
            tmem_alloc(smem_addr(tmem_slot), uint32_t(p.tmem_cols));
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if constexpr (!kWide) griddep_enter(0u);  // kWide: these warps read global memory at their end only
        tmem_base = *tmem_slot;
    }

    if (warp == MMA_WARP) {
        // ============================================================ MMA issuer
        const uint64_t dx = smem_desc(sX16, 16, 1024);
        const uint32_t x_kb = (uint32_t(T) * 128u) >> 4;  // the second 64 of K
        uint32_t c = 0, turn = 0;
        [[maybe_unused]] uint32_t x = 0, x_phase = 0;
        for (int32_t st = st0; st < st1; ++st) {
            if (!__all_sync(0xffffffffu, mbar_wait(ready_bar(c), turn, p.wait))) break;
            if constexpr (kWide) {
                if (!__all_sync(0xffffffffu, mbar_wait(x_full(x), x_phase, p.wait))) break;
            }
            tc_fence_after();
            const uint32_t a0 = tmem_base + uint32_t(acc_cols) + c * lin::I8_A_COLS;
            const uint64_t x0 = dx + (kWide ? x : c) * 2u * x_kb;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // 16 of K each
                mma_f16_tmem_elect(tmem_base, a0 + ks * 8, x0 + (ks / 4) * x_kb + (ks % 4) * 2, p.idesc, st != st0 || ks != 0 ? 1u : 0u);
            mma_commit_elect(used_bar(c));
            turn ^= c;  // two copies in turn
            c ^= 1u;
            if constexpr (kWide) {
                mma_commit_elect(x_empty(x));
                if (++x == uint32_t(XST)) { x = 0; x_phase ^= 1u; }
            }
        }
        // also what the epilogue waits for; after a wait that ran out, no MMA may
        // still be writing TMEM when it is freed
        mma_commit_elect(done_bar);
        __all_sync(0xffffffffu, mbar_wait_slow(done_bar, 0, cleanup_wait(p.wait), false));
    } else if (warp >= EPI_WARP0) {
        // ============================================================ to fp16, then epilogue
        // Two groups of four warps take the stages in turn, so that one's loads and stores
        // pass while the other converts. With an odd number of stages a place in the ring is one
        // group's and then the other's. A wait for a phase tells it from the phase before only, and
        // copies land in any order: a group may come to a place whose earlier copy, the other
        // group's, has not landed, and the phase before that one has the parity it asks for. So it
        // first waits until the other group has released the place.
        const int q = warp & 3, group = ew / 4;  // the TMEM lanes this warp may write
        const uint32_t row = uint32_t(q * 32 + lane), thread = uint32_t(ew & 3) * 32u + uint32_t(lane);
        const uint32_t a_tmem = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(acc_cols);
        const uint32_t tasks = uint32_t(valid) * 8u;  // what lies in the copies of further tokens reaches no row of C
        const uint32_t c = uint32_t(group);  // the group's copy
        uint32_t stage = uint32_t(group), phase = 0, turn = 0;
        bool ok = true;
        for (int32_t st = st0 + group; st < st1; st += 2) {
            if ((NST & 1) != 0 && st >= st0 + NST && !__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, p.wait))) {
                ok = false;
                break;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, p.wait))) {
                ok = false;
                break;
            }
            // the copy's place is free
            if (!__all_sync(0xffffffffu, mbar_wait(used_bar(c), turn ^ 1u, p.wait))) {
                ok = false;
                break;
            }
            tc_fence_after();
            // tokens: 16 bytes of K of one token at a time, four on their way together
            const uint32_t x_from = sX + stage * x_bytes, x_to = sX16 + c * 2u * x_bytes;
#pragma unroll 1
            for (uint32_t e0 = thread; !kWide && e0 < tasks; e0 += 4u * 128u) {
                uint32_t x[4][4];
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const uint32_t e = e0 + k * 128u;
                    if (e < tasks) ld_shared_v4(x_from + swz128(e >> 3, e & 7u), x[k][0], x[k][1], x[k][2], x[k][3]);
                }
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const uint32_t e = e0 + k * 128u;
                    if (e >= tasks) break;
                    const uint32_t r = e >> 3, u = e & 7u, to = x_to + (u >> 2) * x_bytes, v = (u & 3u) * 2u;
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        const uint2 lo = i8x4_to_f16(x[k][2 * i]), hi = i8x4_to_f16(x[k][2 * i + 1]);
                        st_shared_v4(to + swz128(r, v + i), lo.x, lo.y, hi.x, hi.y);
                    }
                }
            }
            uint32_t w[8][4];
            const uint32_t w_row = sW + stage * lin::I8_W_BYTES;
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) ld_shared_v4(w_row + swz128(row, i), w[i][0], w[i][1], w[i][2], w[i][3]);
            if constexpr (!kWide) fence_proxy_async_smem();
            __syncwarp();
            // the stage has been read: its bytes in flight are what the stream's rate goes by
            if (lane == 0) mbar_arrive(empty_bar(stage));
            __syncwarp();  // the stores to tensor memory are the whole warp's
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t a[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint2 f = i8x4_to_f16(w[4 * half + i / 4][i % 4]);
                    a[2 * i] = f.x;
                    a[2 * i + 1] = f.y;
                }
                tmem_st_32x32b_x32(a_tmem + c * lin::I8_A_COLS + 32 * half, a);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready_bar(c));
            stage += 2;
            if (stage >= uint32_t(NST)) { stage -= uint32_t(NST); phase ^= 1u; }
            turn ^= 1u;
        }
        if constexpr (kWide) griddep_wait();  // long over; the loads from here on go through L1
        if (vec) split_columns<true, true>(p, S, rank, ew, lane, m0, n0, valid, columns);
        else split_columns<true, false>(p, S, rank, ew, lane, m0, n0, valid, columns);
        ready = __all_sync(0xffffffffu, mbar_wait(done_bar, 0, p.wait)) && ok;
        tc_fence_after();
    }

    // ---------------------------------------------------------------- the cluster's sum and the epilogue, as in linear_split
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (ready) {
        // two warps per TMEM lane quarter: rows [0, T/2) and [T/2, T) of the tile
        const int q = warp & 3, t0 = (ew / 4) * (T / 2);
        with_split(S, [&](auto s) {
            split_send<decltype(s)::value>(tmem_base + (uint32_t(q * 32) << 16), base, rank, q * 32 + lane, t0, min(t0 + T / 2, valid),
                                           acc_cols);
        });
        tc_fence_before();
    }
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (ready) {
        const bool one = valid <= EPI_WARPS * S;  // a row for each warp at most
        with_split(S, [&](auto s) {
            constexpr int SPLIT = decltype(s)::value;
            if (vec && one) split_rows<true, SPLIT, true, 1>(p, base, rank, ew, lane, m0, n0, valid, columns);
            else if (vec) split_rows<true, SPLIT, true, kSplitRows>(p, base, rank, ew, lane, m0, n0, valid, columns);
            else split_rows<true, SPLIT, false, kSplitRows>(p, base, rank, ew, lane, m0, n0, valid, columns);
        });
    }
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem_base, uint32_t(p.tmem_cols));
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
