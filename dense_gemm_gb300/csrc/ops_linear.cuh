// A product with its epilogue (sm_103a): C = act(s_a s_b (A @ B) + bias) + R,
// fp16 / bf16 / e4m3 operands, fp32 sums, and the elementwise part of its
// backward pass (D = G act'(P) with the column sums of D).
//
// Two kernels:
//   linear_pair   256 x 256 tiles on CTA pairs: the persistent tcgen05 kernel of
//                 gemm_pair.cuh (same rings, roles and tile order; TMA loads,
//                 static order) with an epilogue that works on the tile while it
//                 is in registers. The residual's tile is fetched by TMA into the
//                 buffers the output leaves through, during the main loop.
//   linear_split  few rows or few tiles: 128 columns of C by T rows per CTA with
//                 the product transposed (the weights are the 128-row operand, the
//                 T tokens the N side), K split over a cluster and the partial
//                 sums added through distributed shared memory.
#pragma once
#include "gemm_pair.cuh"
#include "ops_norm.cuh"

namespace g16 {

// ------------------------------------------------------------------ 8-bit tensor-core products
// kind::f8f6f4 with both operands e4m3: K = 32 per instruction, 32 bytes as
// kind::f16's K = 16, so descriptors and steps are the same.
__device__ __forceinline__ void mma_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred pe, pa;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "setp.ne.b32 pa, %4, 0;\n\t"
        "@pe tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, pa;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_f8_pair_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred pe, pa;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "setp.ne.b32 pa, %4, 0;\n\t"
        "@pe tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, pa;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// ------------------------------------------------------------------ activations
// Exponentials are 2^(x log2 e) by ex2.approx (2 units in the last place, plus the
// argument's rounding) and reciprocals rcp.approx (1): silu and the tanh form of gelu
// are relatively within (8 + 2 |x|) and (8 + 8 |z|) 2^-24, z the logistic's argument,
// inside the 16-bit outputs' rounding. Work is on pairs of values, one
// instruction per pair where there is one (fma2 and its like).
// The normal distribution's cumulative function Phi is Abramowitz & Stegun 26.2.17: for
// x >= 0, 1 - Z(x) (b1 t + ... + b5 t^5) with t = 1 / (1 + 0.2316419 x) and Z the
// density, which gelu's slope needs too. It is off by less than 7.5e-8, absolutely, so
// gelu by 7.5e-8 |x|. Relatively that grows in the negative tail, where Phi itself is
// small: 5e-5 at x = -3 (gelu -0.004), 4.7e-4 at -4 (-1.3e-4), 1.6e-3 at -5 (-1.4e-6),
// 3.6e-3 at -6 (-6e-9): from -5 on about half a unit of a bf16 value, more in fp16 or
// fp32. (1 + erf(x / sqrt 2) in fp32 cancels there and is 0 from -5.5 on.) A logistic
// below 2^-126 is 0.
// D = G gelu'(P) of 4096 x 8192 takes 82 us with CUDA's erff and __expf, 57 with the
// formula value by value, 36.5 in pairs with four rows loaded ahead.
constexpr uint32_t kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;  // GEMM_ACT_*
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, v); }
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 exp2_approx(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_approx(float2 x) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(x.y));
    return r;
}

// 1 / (1 + exp(-z))
__device__ __forceinline__ float2 logistic(float2 z) {
    return rcp_approx(add2(pair_of(1.0f), exp2_approx(mul2(z, pair_of(-kLog2E)))));
}

__device__ __forceinline__ void normal_parts(float2 x, float2 &cdf, float2 &density) {
    density = mul2(exp2_approx(mul2(mul2(x, x), pair_of(-0.5f * kLog2E))), pair_of(kInvSqrt2Pi));
    const float2 t = rcp_approx(fma2(make_float2(fabsf(x.x), fabsf(x.y)), pair_of(0.2316419f), pair_of(1.0f)));
    float2 q = fma2(t, pair_of(1.330274429f), pair_of(-1.821255978f));
    q = fma2(t, q, pair_of(1.781477937f));
    q = fma2(t, q, pair_of(-0.356563782f));
    q = fma2(t, q, pair_of(0.319381530f));
    q = mul2(mul2(q, t), density);
    const float2 above = fma2(q, pair_of(-1.0f), pair_of(1.0f));
    cdf = make_float2(x.x < 0.0f ? q.x : above.x, x.y < 0.0f ? q.y : above.y);
}

// z with gelu's tanh form = x / (1 + exp(-z))
__device__ __forceinline__ float2 tanh_argument(float2 x) {
    const float2 x2 = mul2(x, x);
    return mul2(mul2(x, pair_of(kTwoSqrt2OverPi)), fma2(x2, pair_of(0.044715f), pair_of(1.0f)));
}

template <uint32_t ACT>
__device__ __forceinline__ float2 act_value(float2 x) {
    if constexpr (ACT == kActRelu) {
        return make_float2(x.x < 0.0f ? 0.0f : x.x, x.y < 0.0f ? 0.0f : x.y);
    } else if constexpr (ACT == kActSilu) {
        return mul2(x, logistic(x));
    } else if constexpr (ACT == kActGelu) {
        float2 cdf, density;
        normal_parts(x, cdf, density);
        return mul2(x, cdf);
    } else if constexpr (ACT == kActGeluTanh) {
        return mul2(x, logistic(tanh_argument(x)));
    } else {
        return x;
    }
}

template <uint32_t ACT>
__device__ __forceinline__ float2 act_slope(float2 x) {
    if constexpr (ACT == kActRelu) {
        return make_float2(x.x > 0.0f ? 1.0f : 0.0f, x.y > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (ACT == kActSilu) {  // s + x s (1 - s)
        const float2 s = logistic(x), xs = mul2(x, s);
        return fma2(xs, fma2(s, pair_of(-1.0f), pair_of(1.0f)), s);
    } else if constexpr (ACT == kActGelu) {
        float2 cdf, density;
        normal_parts(x, cdf, density);
        return fma2(x, density, cdf);
    } else if constexpr (ACT == kActGeluTanh) {  // s + x s (1 - s) z'
        const float2 s = logistic(tanh_argument(x)), xs = mul2(x, s);
        const float2 dz = fma2(mul2(x, x), pair_of(0.134145f * kTwoSqrt2OverPi), pair_of(kTwoSqrt2OverPi));
        return fma2(mul2(xs, fma2(s, pair_of(-1.0f), pair_of(1.0f))), dz, s);
    } else {
        return pair_of(1.0f);
    }
}

template <uint32_t ACT, int N>
__device__ __forceinline__ void act_all(float (&x)[N]) {
    static_assert(N % 2 == 0, "pairs");
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 v = act_value<ACT>(make_float2(x[i], x[i + 1]));
        x[i] = v.x;
        x[i + 1] = v.y;
    }
}

template <int N>
__device__ __forceinline__ void apply_act(uint32_t act, float (&x)[N]) {
    switch (act) {  // uniform
        case kActRelu: act_all<kActRelu>(x); break;
        case kActGelu: act_all<kActGelu>(x); break;
        case kActGeluTanh: act_all<kActGeluTanh>(x); break;
        case kActSilu: act_all<kActSilu>(x); break;
        default: break;
    }
}

// ------------------------------------------------------------------ elements by run-time type (0 fp32, 1 fp16, 2 bf16)
__device__ __forceinline__ float load_elem(const void *p, uint32_t type, int64_t at) {
    if (type == 0) return static_cast<const float *>(p)[at];
    if (type == 1) return __half2float(static_cast<const __half *>(p)[at]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]);
}

__device__ __forceinline__ void store_elem(void *p, uint32_t type, int64_t at, float v) {
    if (type == 0) static_cast<float *>(p)[at] = v;
    else if (type == 1) static_cast<__half *>(p)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float2 unpack_16x2(uint32_t w, uint32_t type) {
    if (type == 1) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// ------------------------------------------------------------------ parameters
struct EpilogueParams {
    void *c;
    const void *r;  // nullptr: no residual
    void *pre;      // nullptr: not stored
    const void *bias;
    const float *sa, *sb;
    int64_t ldc, ldr, ldp;
    uint32_t type;       // of C, residual and pre
    uint32_t bias_type;
    uint32_t act;
    uint32_t c_tma, r_tma, p_tma;  // described by a tensor map (linear_pair)
    uint32_t vec4;                 // four consecutive columns of C, R and pre are aligned to their size together
};

// How one operand's part of a stage is fetched. Issuing a copy costs its warp some
// hundred cycles, and more when the operands of the instruction are not uniform
// over the warp, so each operand has a producer warp of its own and, where that is
// possible, a stage is one copy, issued by an elected lane from uniform values:
// kLoadOne is a box of a two-dimensional map. kLoadBoxed brings several pieces, the
// k-blocks of a stage one after the other (K-major) or the 64-wide chunks
// (MN-major), through a third dimension of the map; that needs rows that are a
// multiple of the piece, since the third dimension would run into the next row
// otherwise. kLoadLanes issues each piece from a lane of its own.
constexpr uint32_t kLoadOne = 0, kLoadBoxed = 1, kLoadLanes = 2;
struct OperandLoad {
    uint32_t mn;    // 1: MN-major in memory and in shared memory
    uint32_t mode;  // kLoad*
    int32_t copies;  // kLoadLanes: pieces of a stage
};

// kPair: counted on an mbarrier of the pair's CTA 0 (shared::cluster address).
template <bool kPair>
__device__ __forceinline__ void tma_load_2d_elect(uint32_t dst, const void *tmap, int32_t x, int32_t y, uint32_t bar) {
    if (!G16_CHECK((x & 7) == 0 && smem_window_ok(dst, 16))) return;
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(tmap), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(tmap), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tma_load_3d_elect(uint32_t dst, const void *tmap, int32_t x, int32_t y, int32_t z, uint32_t bar) {
    if (!G16_CHECK((x & 7) == 0 && smem_window_ok(dst, 16))) return;
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
            "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
            "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void mbar_expect_tx_elect(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred pe;\n\t"
        "elect.sync _|pe, 0xffffffff;\n\t"
        "@pe mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
        : "memory");
}

// The copies of the stage that starts at k-block kb (of `be` elements), for the
// rows or columns from `mn` on. Whole warp; pieces lie `piece` bytes apart.
template <uint32_t MODE, bool kMn, bool kPair>
__device__ __forceinline__ void issue_copies(const CUtensorMap *map, uint32_t dst, uint32_t piece, int32_t copies, int32_t kb,
                                             int32_t be, int32_t mn, uint32_t bar, int lane) {
    const int32_t k0 = kb * be;
    if constexpr (MODE == kLoadOne) {
        tma_load_2d_elect<kPair>(dst, map, kMn ? mn : k0, kMn ? k0 : mn, bar);
    } else if constexpr (MODE == kLoadBoxed) {
        tma_load_3d_elect<kPair>(dst, map, 0, kMn ? k0 : mn, kMn ? mn / MN_CHUNK : kb, bar);
    } else if (lane < copies) {
        const int32_t x = kMn ? mn + lane * MN_CHUNK : k0 + lane * be, y = kMn ? k0 : mn;
        if constexpr (kPair) tma_load_2d_pair(dst + uint32_t(lane) * piece, map, x, y, bar);
        else tma_load_2d(dst + uint32_t(lane) * piece, map, x, y, bar);
    }
}

// Asks for the same copies' lines in L2 only. Nothing is read by it, so it may come
// before the kernel that the launch depends on has ended: a line that is written
// after all is written in L2. (kLoadLanes: not worth its code.)
template <uint32_t MODE, bool kMn>
__device__ __forceinline__ void prefetch_copies(const CUtensorMap *map, int32_t kb, int32_t be, int32_t mn) {
    const int32_t k0 = kb * be;
    if constexpr (MODE == kLoadOne) {
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}" ::"l"(map),
            "r"(kMn ? mn : k0), "r"(kMn ? k0 : mn)
            : "memory");
    } else if constexpr (MODE == kLoadBoxed) {
        asm volatile(
            "{\n\t.reg .pred pe;\n\t"
            "elect.sync _|pe, 0xffffffff;\n\t"
            "@pe cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}" ::"l"(map),
            "r"(0), "r"(kMn ? k0 : mn), "r"(kMn ? mn / MN_CHUNK : kb)
            : "memory");
    }
}

// Calls f with the mode and the major-ness as template arguments.
template <typename F>
__device__ __forceinline__ void with_load(const OperandLoad &o, F f) {
    using std::integral_constant;
    using One = integral_constant<uint32_t, kLoadOne>;
    using Boxed = integral_constant<uint32_t, kLoadBoxed>;
    using Lanes = integral_constant<uint32_t, kLoadLanes>;
    if (o.mn) {
        if (o.mode == kLoadBoxed) f(Boxed(), std::true_type());
        else if (o.mode == kLoadOne) f(One(), std::true_type());
        else f(Lanes(), std::true_type());
    } else {
        if (o.mode == kLoadBoxed) f(Boxed(), std::false_type());
        else if (o.mode == kLoadOne) f(One(), std::false_type());
        else f(Lanes(), std::false_type());
    }
}

struct LinearParams {
    int64_t M, N;
    Sched sched;
    int32_t num_kb;
    OperandLoad a, b, b_half;  // b_half: linear_pair's half tiles
    uint32_t idesc;
    // linear_pair: units below `whole` are tiles; from there on, halves (128
    // columns) of the tiles `whole`, whole + 1, ...
    int32_t num_units, whole;
    uint32_t idesc_half;
    int32_t stages, bufs;     // linear_pair: ring depth, staging buffers per epilogue warp
    int32_t T, tmem_cols;     // linear_split: rows of C per CTA, TMEM columns
    int32_t split;            // linear_split: CTAs of a cluster along K
    uint32_t late;            // griddep_enter
    EpilogueParams e;
    WaitCtl wait;
};

// ================================================================== linear_pair
namespace lin {
constexpr int PAIR_STAGES = 6;  // at most; 5 when two staging buffers per warp are needed
constexpr int STAGE_BYTES = pair::A_STAGE_BYTES + pair::B_STAGE_BYTES;
constexpr int PAIR_THREADS = (3 + EPI_WARPS) * 32;  // A's and B's producers, MMA, epilogue
constexpr int BUF_BYTES = 4096;  // 32 rows of 128 bytes
// full[6], empty[6], tfull[2], tempty[2], tdone[2], drain, residual[8 warps][2]
constexpr int PAIR_BARS = 2 * PAIR_STAGES + 3 * NUM_ACC + 1 + 2 * EPI_WARPS;
constexpr int ring_and_staging(int stages, int bufs) { return stages * STAGE_BYTES + bufs * EPI_WARPS * BUF_BYTES; }
constexpr int PAIR_RING = ring_and_staging(6, 1);
static_assert(ring_and_staging(5, 2) == PAIR_RING, "one shared-memory size for both shapes");
constexpr int PAIR_OFF_BAR = PAIR_RING;
constexpr int PAIR_OFF_SLOT = PAIR_OFF_BAR + PAIR_BARS * 8;
constexpr int PAIR_SMEM = PAIR_OFF_SLOT + 16 + 1024;
static_assert(PAIR_SMEM <= 232448, "exceeds the 227 KiB per-CTA shared memory limit");
}  // namespace lin

// A unit of linear_pair: the first row and column of this CTA's part of the
// output and the unit's columns (256, or 128 for half a tile).
struct Unit {
    int64_t row0, col0;
    int32_t cols;
};
__device__ __forceinline__ Unit unit_of(const LinearParams &p, int32_t u, uint32_t rank) {
    const bool half = u >= p.whole;
    const int32_t v = u - p.whole;
    int32_t tm, tn;
    tile_coords(half ? p.whole + (v >> 1) : u, p.sched, tm, tn);
    return Unit{int64_t(tm) * pair::TILE_M + int64_t(rank) * pair::CTA_M,
                int64_t(tn) * pair::TILE_N + (half && (v & 1) ? pair::TILE_N / 2 : 0), half ? pair::TILE_N / 2 : pair::TILE_N};
}

// The epilogue of one warp: 32 rows (TMEM lanes) by half the unit's columns.
// OB: bytes per element of C. A chunk is 128 bytes of each row; the warp's chunks
// take its staging buffers in turn. kScaled: rows and columns have factors.
template <bool kScaled, int OB>
struct PairEpilogue {
    static constexpr int CHUNK = 128 / OB;  // columns: 64 or 32
    const LinearParams &p;
    const CUtensorMap *tmC, *tmR, *tmP;
    uint32_t stg, rbar;  // this warp's staging buffers and residual barriers (2)
    int lane, q, half;   // TMEM lane quarter, column half
    uint32_t rank;
    int32_t next_u, next_c, step;  // the next chunk to fetch the residual of; units between this CTA's
    uint32_t fetched, used;        // residual chunks asked for and taken

    __device__ __forceinline__ uint32_t buf(uint32_t b) const { return stg + b * lin::BUF_BYTES; }
    __device__ __forceinline__ bool prefetches() const { return p.e.r != nullptr && p.e.r_tma; }

    // The buffer of the n-th residual chunk, where C's will be (with pre that is the
    // second one), and the phase of its barrier. (Plain loads next to pre, instead:
    // 8192 x 8192 x 128 499 us, so 102.)
    __device__ __forceinline__ bool in_turns() const { return p.bufs == 2 && p.e.pre == nullptr; }
    __device__ __forceinline__ uint32_t residual_buf(uint32_t n) const { return p.e.pre != nullptr ? 1u : in_turns() ? n & 1u : 0u; }
    __device__ __forceinline__ uint32_t residual_phase(uint32_t n) const { return (in_turns() ? n >> 1 : n) & 1u; }

    // Start fetching the residual's 32 rows x CHUNK columns of the next chunk that
    // has not been asked for into its buffer (whole warp).
    __device__ __forceinline__ void fetch_residual() {
        if (next_u >= p.num_units) return;
        const Unit u = unit_of(p, next_u, rank);
        if (lane == 0) {
            const uint32_t b = residual_buf(fetched);
            mbar_arrive_expect_tx(rbar + 8u * b, lin::BUF_BYTES);
            tma_load_2d(buf(b), tmR, int32_t(u.col0) + half * (u.cols / 2) + next_c * CHUNK, int32_t(u.row0) + q * 32, rbar + 8u * b);
        }
        ++fetched;
        if (++next_c * CHUNK == u.cols / 2) {
            next_c = 0;
            next_u += step;
        }
    }

    // Buffer b <- the residual's 32 rows x CHUNK columns, with plain loads. Places
    // past the last row or column get its value, which goes nowhere: without
    // conditions, and with a batch's loads before its first store to shared memory,
    // they are in flight together (8192 x 8191 x 128: row by row 440 us, so 183).
    __device__ __forceinline__ void load_residual(uint32_t b, int64_t row0, int64_t col0) {
        constexpr int PER_LANE = CHUNK / 32, BATCH = 16;
        const int64_t last = p.N - 1, c = col0 + PER_LANE * lane;
        const int64_t at0 = c < last ? c : last, at1 = c + 1 < last ? c + 1 : last;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += BATCH) {
            uint32_t w[BATCH], hi[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int64_t r = row0 + r0 + i, at = (r < p.M ? r : p.M - 1) * p.e.ldr;
                if constexpr (OB == 4) {
                    w[i] = static_cast<const uint32_t *>(p.e.r)[at + at0];
                } else {
                    w[i] = static_cast<const uint16_t *>(p.e.r)[at + at0];
                    hi[i] = static_cast<const uint16_t *>(p.e.r)[at + at1];
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if constexpr (OB == 2) w[i] |= hi[i] << 16;
                st_shared_s32(buf(b) + swz128(r0 + i, lane >> 2) + (lane & 3) * 4, int32_t(w[i]));
            }
        }
        __syncwarp();
    }

    // Buffer b -> 32 rows x CHUNK columns of `dst`, by TMA or plain stores.
    __device__ __forceinline__ void store(uint32_t b, void *dst, int64_t ld, const CUtensorMap *map, bool tma, int64_t row0,
                                          int64_t col0) {
        if (tma) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (row0 < p.M && col0 < p.N)
                    tma_store_2d_hint(map, buf(b), int32_t(col0), int32_t(row0), l2_policy_evict_normal());
                bulk_commit_group();
            }
            return;
        }
        __syncwarp();
        const int64_t rows = p.M - row0;
        constexpr int PER_LANE = CHUNK / 32;
        const int64_t col = col0 + PER_LANE * lane;
        if (col < p.N) {
            constexpr int BATCH = 8;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += BATCH) {
                uint32_t w[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) w[i] = ld_shared_b32(buf(b) + swz128(r0 + i, lane >> 2) + (lane & 3) * 4);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int r = r0 + i;
                    if (r >= rows || !G16_CHECK(row0 + r < p.M && col >= 0)) continue;
                    if constexpr (OB == 4) {
                        static_cast<uint32_t *>(dst)[(row0 + r) * ld + col] = w[i];
                    } else {
                        uint16_t *d = static_cast<uint16_t *>(dst) + (row0 + r) * ld + col;
                        d[0] = uint16_t(w[i] & 0xffffu);
                        if (col + 1 < p.N) d[1] = uint16_t(w[i] >> 16);
                    }
                }
            }
        }
        __syncwarp();  // every lane has read the buffer
        fence_proxy_async_smem();  // before a TMA fetch writes it
    }

    // x -> this lane's row of buffer b; `part`: which 32 columns of a 16-bit chunk
    __device__ __forceinline__ void put(uint32_t b, int part, const float (&x)[32]) {
        if constexpr (OB == 4) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                st_shared_v4(buf(b) + swz128(lane, u), __float_as_uint(x[4 * u]), __float_as_uint(x[4 * u + 1]),
                             __float_as_uint(x[4 * u + 2]), __float_as_uint(x[4 * u + 3]));
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                st_shared_v4(buf(b) + swz128(lane, 4 * part + u), pack_16x2(x[8 * u], x[8 * u + 1], p.e.type),
                             pack_16x2(x[8 * u + 2], x[8 * u + 3], p.e.type),
                             pack_16x2(x[8 * u + 4], x[8 * u + 5], p.e.type),
                             pack_16x2(x[8 * u + 6], x[8 * u + 7], p.e.type));
        }
    }

    __device__ __forceinline__ void add_residual(uint32_t b, int part, float (&x)[32]) {
        if constexpr (OB == 4) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                uint32_t w[4];
                ld_shared_v4(buf(b) + swz128(lane, u), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * u + i] += __uint_as_float(w[i]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t w[4];
                ld_shared_v4(buf(b) + swz128(lane, 4 * part + u), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack_16x2(w[i], p.e.type);
                    x[8 * u + 2 * i] += f.x;
                    x[8 * u + 2 * i + 1] += f.y;
                }
            }
        }
    }

    // One unit's part of this warp: rows row0 .. row0 + 31, `groups` (4 or 2) times
    // 32 columns from col0 on. False if a wait ran out.
    // Two 32-column turns are unrolled, not four: the code of five activations in
    // each is fetched more slowly than it runs (1024 x 4096 x 1024: 13.9 us with
    // four, 11.6 with two and the set-up before griddep_enter).
    template <typename Drained>
    __device__ __forceinline__ bool unit(uint32_t t_addr, int64_t row0, int64_t col0, int groups, const float (&bias)[4],
                                         const float (&sb)[4], float sa, Drained drained) {
        const bool has_r = p.e.r != nullptr, has_p = p.e.pre != nullptr, pref = prefetches();
        const bool two = p.bufs == 2;
        bool ok = true;
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(t_addr, v[0]);
#pragma unroll 2
        for (int j = 0; j < groups; ++j) {
            const int i0 = j & 1, j0 = j - i0;
            const int c = j * 32 / CHUNK;
            const int part = OB == 4 ? 0 : i0;  // which 32 columns of a 16-bit chunk
            // C's buffer: with pre, 0 is pre's; chunks of a unit come in pairs except for
            // half a tile in 16 bits, so with prefetches the count of chunks decides
            const uint32_t b = has_p ? 1u : !two ? 0u : pref ? residual_buf(used) : uint32_t(c & 1);
            tmem_ld_wait();
            if (j + 1 < groups) tmem_ld_32x32b_x32(t_addr + (j + 1) * 32, v[i0 ^ 1]);
            else drained();
            if (part == 0) {  // the buffers of a new chunk
                if (pref) {
                    if (!__all_sync(0xffffffffu, mbar_wait(rbar + 8u * b, residual_phase(used), p.wait))) ok = false;
                } else {
                    // the buffer's previous store has read it
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
                    if (has_r) load_residual(b, row0, col0 + c * CHUNK);
                }
            }
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i0][i]);
            if constexpr (kScaled) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= sa * __shfl_sync(0xffffffffu, j0 == 0 ? sb[i0] : sb[i0 + 2], i);
            }
            if (p.e.bias != nullptr) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] += __shfl_sync(0xffffffffu, j0 == 0 ? bias[i0] : bias[i0 + 2], i);
            }
            if (has_p) put(0, part, x);
            apply_act(p.e.act, x);
            if (has_r) add_residual(b, part, x);
            put(b, part, x);
            if (part == (OB == 4 ? 0 : 1)) {
                if (has_p) store(0, p.e.pre, p.e.ldp, tmP, p.e.p_tma != 0, row0, col0 + c * CHUNK);
                store(b, p.e.c, p.e.ldc, tmC, p.e.c_tma != 0, row0, col0 + c * CHUNK);
                if (pref) {  // this buffer takes the next chunk, or in turns the one after
                    ++used;
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
                    if (ok) fetch_residual();
                }
            }
        }
        return ok;
    }

    // Before the first unit.
    __device__ __forceinline__ void begin() {
        if (!prefetches()) return;
        fetch_residual();
        if (in_turns()) fetch_residual();
    }

    // After the last unit, or after a wait ran out: no copy may still be on its
    // way into or out of this warp's buffers when the CTA ends.
    __device__ __forceinline__ void end() {
        for (; used < fetched; ++used)
            mbar_wait_slow(rbar + 8u * residual_buf(used), residual_phase(used), cleanup_wait(p.wait), false);
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }
};

// Bound by the tensor cores, over many rounds of tiles by the clock the power limit
// leaves: 8192 x 16384 x 4096 bf16 with gelu and pre 596 us (1.85 PFLOP/s) a call in
// short runs, 617 to 690 in long ones; 4096 x 8192 x 8192 e4m3 145 us (3.78 PFLOP/s).
// Where tiles fill few rounds, by what a tile costs around its k-blocks (4000 x 5000
// x 3000, 4.2 rounds: 95 us, tensor pipe 61 % active) and, with halves, by what L2
// delivers (512 x 4096 x 4096: 0.22 us a k-block, 14 TB/s, for 0.12 us of products; 8
// stages instead of 6 change nothing). Two staging buffers per warp instead of one
// only where the residual or pre needs them: the sixth stage is worth more (8192 x
// 8192 x 4096: 315 us with one buffer, 340 with two and 5 stages).
// kScaled without kF8: whole numbers as fp16, with the scales of 8-bit integers.
template <bool kF8, int OB, bool kScaled = kF8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lin::PAIR_THREADS, 1)
    linear_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmBhalf, const __grid_constant__ CUtensorMap tmC,
                const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmP, const LinearParams p) {
    constexpr int MAXST = lin::PAIR_STAGES;
    constexpr int BKE = kF8 ? 128 : 64;  // K per stage, elements
    constexpr int MMA_WARP = 1, EPI_WARP0 = 2, B_WARP = EPI_WARP0 + EPI_WARPS;
    const int NST = p.stages;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // same offset in both CTAs
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t sA = base;
    const uint32_t sB = base + uint32_t(NST) * pair::A_STAGE_BYTES;
    const uint32_t sE = base + uint32_t(NST) * lin::STAGE_BYTES;
    const uint32_t bar0 = base + lin::PAIR_OFF_BAR;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (MAXST + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * MAXST + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * MAXST + NUM_ACC + a); };
    auto tdone_bar = [&](int a) { return bar0 + 8u * (2 * MAXST + 2 * NUM_ACC + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * MAXST + 3 * NUM_ACC);
    const uint32_t res_bar0 = drain_bar + 8u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + lin::PAIR_OFF_SLOT);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0: issues the MMAs
    const int32_t pair_id = int32_t(blockIdx.x >> 1);
    const int32_t num_pairs = int32_t(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < MAXST; ++s) {
            mbar_init(full_bar(s), 1);   // CTA 0's arrive.expect_tx, both CTAs' bytes
            mbar_init(empty_bar(s), 1);  // CTA 0's MMA commit (multicast)
        }
        for (int a = 0; a < NUM_ACC; ++a) {
            mbar_init(tfull_bar(a), 1);               // CTA 0's MMA commit (multicast)
            mbar_init(tempty_bar(a), EPI_WARPS + 1);  // CTA 0's epilogue warps, CTA 1's relay
            mbar_init(tdone_bar(a), EPI_WARPS);       // this CTA's epilogue warps
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(res_bar0 + 8u * i, 1);
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {  // one warp in each CTA of the pair, collectively
        tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) prefetch_tensormap(&tmA);
    if (warp == B_WARP && lane == 0) {
        prefetch_tensormap(&tmB);
        if (p.whole < p.num_units) prefetch_tensormap(&tmBhalf);
    }
    if (warp == EPI_WARP0 && lane == 0) {
        if (p.e.c_tma) prefetch_tensormap(&tmC);
        if (p.e.r_tma) prefetch_tensormap(&tmR);
        if (p.e.p_tma) prefetch_tensormap(&tmP);
    }
    tc_fence_before();
    cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
    tc_fence_after();
    // Each role waits for the previous kernel on the stream (griddep_enter) right
    // before its first access to global memory: by then its parameters are read and
    // its code is fetched, which took 1.4 us between the wait and the first copy.
    const uint32_t tmem_base = *tmem_slot;
    const int32_t num_kb = p.num_kb;

    if (warp == 0 || warp == B_WARP) {
        // ============================================================ producers (both CTAs)
        // One warp per operand; A's announces a stage's bytes (both operands', both
        // CTAs') on CTA 0's barrier. Copies may land before the announcement: a phase
        // ends only after it.
        uint32_t stage = 0, phase = 0, issued = 0;
        bool ok = true;
        const bool is_a = warp == 0;
        // All k-blocks of one unit; what does not change over them is a template argument.
        auto load_unit = [&](const Unit &un, const CUtensorMap *map, auto mode, auto mn_major, auto announces, uint32_t tx) {
            const int32_t mn = is_a ? int32_t(un.row0) : int32_t(un.col0) + int32_t(rank) * (un.cols / 2);
            const int32_t copies = is_a ? p.a.copies : un.cols == pair::TILE_N ? p.b.copies : p.b_half.copies;
            const uint32_t s0 = is_a ? sA : sB;
            for (int32_t kb = 0; kb < num_kb; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, p.wait))) {
                    ok = false;
                    break;
                }
                if constexpr (decltype(announces)::value) mbar_expect_tx_elect(full_bar(stage), tx);
                issue_copies<decltype(mode)::value, decltype(mn_major)::value, true>(
                    map, s0 + stage * pair::A_STAGE_BYTES, MN_CHUNK_BYTES, copies, kb, BKE, mn, mapa_shared(full_bar(stage), 0), lane);
                ++issued;
                if (++stage == uint32_t(NST)) { stage = 0; phase ^= 1u; }
            }
        };
        static_assert(pair::A_STAGE_BYTES == pair::B_STAGE_BYTES, "one stage pitch for both operands");
        constexpr uint32_t TX_HALF = 2u * (pair::A_STAGE_BYTES + pair::B_STAGE_BYTES / 2);
        int32_t u = pair_id;
        Unit un = unit_of(p, u, rank);
        bool entered = false;
        auto enter = [&] {
            if (!entered) griddep_enter(p.late);
            entered = true;
        };
        auto next = [&] {
            u += num_pairs;
            if (u < p.num_units) un = unit_of(p, u, rank);
        };
        if (is_a) {
            with_load(p.a, [&](auto mode, auto mn_major) {
                auto all = [&](auto announces) {
                    enter();
                    for (; ok && u < p.num_units; next())
                        load_unit(un, &tmA, mode, mn_major, announces, u < p.whole ? pair::PAIR_TX_BYTES : TX_HALF);
                };
                if (rank == 0) all(std::true_type());
                else all(std::false_type());
            });
        } else {
            if (u < p.whole)
                with_load(p.b, [&](auto mode, auto mn_major) {
                    enter();
                    for (; ok && u < p.whole; next()) load_unit(un, &tmB, mode, mn_major, std::false_type(), 0u);
                });
            if (u < p.num_units)
                with_load(p.b_half, [&](auto mode, auto mn_major) {
                    enter();
                    for (; ok && u < p.num_units; next()) load_unit(un, &tmBhalf, mode, mn_major, std::false_type(), 0u);
                });
        }
        if (!ok && lane == 0) {
            if (rank == 0 && is_a) {
                // Let the copies counted on this CTA's barriers land before exiting.
                const uint32_t n = issued < uint32_t(NST) ? issued : uint32_t(NST);
                for (uint32_t q = issued - n; q < issued; ++q)
                    mbar_wait_slow(full_bar(q % NST), (q / NST) & 1u, cleanup_wait(p.wait), false);
            } else {
                // Copies issued by the other producers are not known here, and CTA 1's count
                // on CTA 0's barriers, which it cannot wait on; give copies already issued
                // time to land (16 KiB reads, microseconds at most).
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        griddep_enter(p.late);
        if (rank == 1) {
            // ======================================================== relay (CTA 1)
            // One release at cluster scope per tile tells CTA 0 that all of this CTA's
            // epilogue warps have drained the accumulator.
            int32_t it = 0;
            for (int32_t u = pair_id; u < p.num_units; u += num_pairs, ++it) {
                const uint32_t acc = it & 1;
                if (!__all_sync(0xffffffffu, mbar_wait(tdone_bar(acc), (uint32_t(it) >> 1) & 1u, p.wait))) break;
                if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
                __syncwarp();
            }
        } else {
            // ======================================================== MMA issuer (CTA 0)
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            int32_t it = 0;
            const DescStep da = make_desc_step(sA, p.a.mn, pair::A_STAGE_BYTES);
            const DescStep db = make_desc_step(sB, p.b.mn, pair::B_STAGE_BYTES);
            for (int32_t u = pair_id; ok && u < p.num_units; u += num_pairs, ++it) {
                const uint32_t idesc = u < p.whole ? p.idesc : p.idesc_half;
                const uint32_t acc = it & 1, use = it >> 1;
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(tempty_bar(acc), (use & 1u) ^ 1u, p.wait))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * pair::TILE_N;
                for (int32_t kb = 0; kb < num_kb; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, p.wait))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a0 = da.base + stage * da.stage;
                    const uint64_t b0 = db.base + stage * db.stage;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {  // 32 bytes of K each
                        if constexpr (kF8)
                            mma_f8_pair_elect(d_tmem, a0 + ks * da.k16, b0 + ks * db.k16, idesc, (kb | ks) != 0 ? 1u : 0u);
                        else
                            mma_f16_pair_elect(d_tmem, a0 + ks * da.k16, b0 + ks * db.k16, idesc, (kb | ks) != 0 ? 1u : 0u);
                    }
                    mma_commit_pair_mc_elect(empty_bar(stage), 0x3);  // both CTAs' slots reusable
                    if (++stage == uint32_t(NST)) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                mma_commit_pair_mc_elect(tfull_bar(acc), 0x3);  // both halves of the tile complete
            }
            mma_commit_pair_elect(drain_bar);
            __all_sync(0xffffffffu, mbar_wait_slow(drain_bar, 0, cleanup_wait(p.wait), false));
        }
    } else {
        // ============================================================ epilogue (both CTAs)
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int ew = warp - EPI_WARP0;
        const int half = ew / 4;  // columns [128 half, 128 half + 128) of the tile
        PairEpilogue<kScaled, OB> ep{p,    &tmC, &tmR, &tmP,    sE + uint32_t(ew) * uint32_t(p.bufs) * lin::BUF_BYTES,
                                 res_bar0 + 16u * ew, lane, q, half, rank, pair_id, 0, num_pairs, 0, 0};
        griddep_enter(p.late);
        ep.begin();
        int32_t it = 0;
        for (int32_t u = pair_id; u < p.num_units; u += num_pairs, ++it) {
            const uint32_t acc = it & 1, use = it >> 1;
            const Unit un = unit_of(p, u, rank);
            const int32_t first = half * (un.cols / 2);  // this warp's first column of the unit
            const int64_t row0 = un.row0 + q * 32, col0 = un.col0 + first;
            const int groups = un.cols / 64;
            // column factors and the row's, one column of each 32 per lane
            float bias[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {1.f, 1.f, 1.f, 1.f}, sa = 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = col0 + 32 * j + lane;
                if (j < groups && col < p.N) {
                    if (p.e.bias != nullptr) bias[j] = load_elem(p.e.bias, p.e.bias_type, col);
                    if (kScaled) sb[j] = p.e.sb[col];
                }
            }
            if (kScaled && row0 + lane < p.M) sa = p.e.sa[row0 + lane];
            if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(acc), use & 1u, p.wait))) break;
            tc_fence_after();
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(tdone_bar(acc));
                    if (rank == 0) mbar_arrive(tempty_bar(acc));  // the MMA warp is in this CTA
                }
            };
            if (!ep.unit(tmem_base + (uint32_t(q * 32) << 16) + acc * pair::TILE_N + first, row0, col0, groups, bias, sb, sa,
                         release))
                break;
        }
        ep.end();
    }

    // ---------------------------------------------------------------- teardown
    griddep_leave(p.late);
    tc_fence_before();
    cluster_sync();  // no CTA leaves while its peer may still use its smem or barriers
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ================================================================== linear_split
namespace lin {
constexpr int SPLIT_THREADS = (2 + EPI_WARPS) * 32;
constexpr int SPLIT_ROWS = 128;                     // columns of C per CTA (TMEM lanes)
constexpr int KPS = 2;                              // k-blocks per stage
constexpr int W_STAGE_BYTES = KPS * SPLIT_ROWS * 128;  // 32 KiB
constexpr int SPLIT_MAX_STAGES = 3;
constexpr int MAX_SPLIT = 8;
// full[S], empty[S], done
constexpr int SPLIT_BARS = 2 * SPLIT_MAX_STAGES + 1;
constexpr int split_ring(int stages, int T) { return stages * (W_STAGE_BYTES + KPS * T * 128); }
constexpr int split_smem(int stages, int T) { return split_ring(stages, T) + SPLIT_BARS * 8 + 16 + 1024; }
}  // namespace lin

// Stores into the shared memory of a CTA of the cluster.
__device__ __forceinline__ void st_dsmem_b32(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// The epilogue on one value of C.
__device__ __forceinline__ float act_one(uint32_t act, float x) {
    float v[2] = {x, x};
    apply_act(act, v);
    return v[0];
}

// Rows [t, t1) of the tile from TMEM (`t_addr`: this warp's lanes, column 0) to the
// CTAs they belong to: row r to CTA r mod S, place r / S, there [place][source
// CTA][128] floats from `base` on. `col`: this lane's column of the tile.
template <int S>
__device__ __forceinline__ void split_send(uint32_t t_addr, uint32_t base, uint32_t rank, int col, int t, int t1, int tmem_cols) {
    uint32_t to[S];  // place 0 of each CTA, from this one
#pragma unroll
    for (int d = 0; d < S; ++d) to[d] = mapa_shared(base + (rank * lin::SPLIT_ROWS + uint32_t(col)) * 4u, uint32_t(d));
#pragma unroll 1
    for (; t < t1; t += 32) {
        uint32_t v[32];
        const int at = min(t, tmem_cols - 32);  // T = 16: one load of 32 columns holds all
        tmem_ld_32x32b_x32(t_addr + uint32_t(at), v);
        tmem_ld_wait();
        const uint32_t off = uint32_t(at) * (lin::SPLIT_ROWS * 4u);  // at is a multiple of S
        if (at == t && t + 32 <= t1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) st_dsmem_b32(to[i % S] + off + uint32_t(i / S * S * lin::SPLIT_ROWS * 4), v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (at + i >= t && at + i < t1) st_dsmem_b32(to[i % S] + off + uint32_t(i / S * S * lin::SPLIT_ROWS * 4), v[i]);
        }
    }
}

// What an epilogue warp of linear_split holds of its columns and of the residual of
// its first rows: fetched while the products run, since nothing hides the latency
// of a load at the end (200 x 4096 x 8192 with a residual: 24.4 us, so 21.7). A lane
// holds four columns: consecutive ones where C, pre and residual take vectors of
// four (vec), else 32 apart, so that a warp's stores are contiguous either way.
constexpr int kSplitRows = 4;  // rows of a warp at a time
struct SplitColumns {
    float bias[4], sb[4];
    uint32_t r[kSplitRows][4];  // as loaded: two or four words
};

template <bool VEC>
__device__ __forceinline__ int split_col(int lane, int i) {
    return VEC ? lane * 4 + i : lane + 32 * i;
}

// The residual of row m at this lane's columns as it lies in memory, converted only
// where it is added, so that several rows' loads are in flight together. A column
// past the last gets its value, which goes nowhere.
template <bool VEC>
__device__ __forceinline__ void split_residual(const LinearParams &p, int64_t m, int32_t n0, int lane, uint32_t (&r)[4]) {
    const int64_t at = m * p.e.ldr;
    if (VEC && p.e.type != 0) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.e.r) + at + n0 + lane * 4);
        r[0] = w.x, r[1] = w.y;
        return;
    }
    int64_t col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = int64_t(n0) + split_col<VEC>(lane, i);
        col[i] = at + (VEC || c < p.N ? c : p.N - 1);
    }
    if (p.e.type == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = static_cast<const uint32_t *>(p.e.r)[col[i]];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = static_cast<const uint16_t *>(p.e.r)[col[i]];
    }
}

template <bool VEC>
__device__ __forceinline__ void add_split_residual(uint32_t type, const uint32_t (&r)[4], float *x) {
    if (type == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += __uint_as_float(r[i]);
    } else if constexpr (VEC) {
        const float2 a = unpack_16x2(r[0], type), b = unpack_16x2(r[1], type);
        x[0] += a.x, x[1] += a.y, x[2] += b.x, x[3] += b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += unpack_16x2(r[i], type).x;
    }
}

// Warp `ew` of CTA `rank` has rows k S + rank of the tile, k = ew, ew + 8, ...; this
// fetches its columns' factors and the residual of the first kSplitRows of them.
template <bool kScaled, bool VEC>
__device__ __forceinline__ void split_columns(const LinearParams &p, int S, uint32_t rank, int ew, int lane, int32_t m0,
                                              int32_t n0, int valid, SplitColumns &h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t n = int64_t(n0) + split_col<VEC>(lane, i);
        const bool in = VEC || n < p.N;
        h.bias[i] = in && p.e.bias != nullptr ? load_elem(p.e.bias, p.e.bias_type, n) : 0.0f;
        h.sb[i] = kScaled && in ? p.e.sb[n] : 1.0f;
    }
    if (p.e.r == nullptr) return;
#pragma unroll
    for (int u = 0; u < kSplitRows; ++u) {
        const int t = (ew + u * EPI_WARPS) * S + int(rank);
        if (t < valid) split_residual<VEC>(p, int64_t(m0) + t, n0, lane, h.r[u]);
    }
}

// Sums the S partial rows of this warp's rows of C, in rank order, and runs the
// epilogue on them, R rows at a time.
template <bool kScaled, int S, bool VEC, int R>
__device__ __forceinline__ void split_rows(const LinearParams &p, uint32_t base, uint32_t rank, int ew, int lane, int32_t m0,
                                           int32_t n0, int valid, SplitColumns &h) {
    const EpilogueParams &e = p.e;
#pragma unroll 1
    for (int k = ew; k * S + int(rank) < valid; k += R * EPI_WARPS) {
        float x[4 * R], sa[R];
        auto tile_row = [&](int u) { return (k + u * EPI_WARPS) * S + int(rank); };
#pragma unroll
        for (int u = 0; u < R; ++u) sa[u] = kScaled && tile_row(u) < valid ? e.sa[int64_t(m0) + tile_row(u)] : 1.0f;
#pragma unroll
        for (int u = 0; u < R; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * u + i] = 0.0f;
            if (R > 1 && tile_row(u) >= valid) continue;
            const uint32_t row = base + uint32_t((k + u * EPI_WARPS) * S * lin::SPLIT_ROWS) * 4u;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t at = row + uint32_t(s * lin::SPLIT_ROWS) * 4u;
                uint32_t w[4];
                if constexpr (VEC) {
                    ld_shared_v4(at + uint32_t(lane) * 16u, w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = ld_shared_b32(at + uint32_t(split_col<VEC>(lane, i)) * 4u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * u + i] += __uint_as_float(w[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * u + i] = (kScaled ? x[4 * u + i] * (sa[u] * h.sb[i]) : x[4 * u + i]) + h.bias[i];
        }
        auto put = [&](void *dst, int64_t ld) {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (R > 1 && tile_row(u) >= valid) continue;
                const float *v = x + 4 * u;
                const int64_t at = (int64_t(m0) + tile_row(u)) * ld + n0 + split_col<VEC>(lane, 0);
                if constexpr (VEC) {
                    if (e.type == 0)
                        *reinterpret_cast<float4 *>(static_cast<float *>(dst) + at) = make_float4(v[0], v[1], v[2], v[3]);
                    else
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(dst) + at) =
                            make_uint2(pack_16x2(v[0], v[1], e.type), pack_16x2(v[2], v[3], e.type));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n0 + int64_t(split_col<VEC>(lane, i)) < p.N && G16_CHECK(m0 + tile_row(u) < p.M))
                            store_elem(dst, e.type, at + 32 * i, v[i]);
                }
            }
        };
        if (e.pre != nullptr) put(e.pre, e.ldp);
        apply_act(e.act, x);
        if (e.r != nullptr) {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                add_split_residual<VEC>(e.type, h.r[u], x + 4 * u);
                // for the next rows, while these are stored
                const int t = tile_row(u) + R * EPI_WARPS * S;
                if (t < valid) split_residual<VEC>(p, int64_t(m0) + t, n0, lane, h.r[u]);
            }
        }
        put(e.c, e.ldc);
    }
}

// Calls f with S as a template argument.
template <typename F>
__device__ __forceinline__ void with_split(int S, F f) {
    switch (S) {
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        case 4: f(std::integral_constant<int, 4>()); break;
        default: f(std::integral_constant<int, 8>()); break;
    }
}

// Cluster of p.split CTAs (1..8) along x, all on the same tile; CTA r sums the
// pairs of k-blocks r n / split ... (r + 1) n / split of n.
// Bound by the weights' stream from DRAM where N K is large (4 x 16384 x 4096: 134
// MB in 23.3 us, 5.8 TB/s), else by the chain first copy - products - cluster barrier
// - partial rows - sum, 5 us of which hold no stream (one token 4096 x 4096: 33.6 MB
// in 7.9 us; 48 x 4096 x 8192: 68 MB in 14.4 us).
template <bool kF8, bool kScaled = kF8>
__global__ void __launch_bounds__(lin::SPLIT_THREADS, 2)
    linear_split(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinearParams p) {
    constexpr int BKE = kF8 ? 128 : 64;
    constexpr int MMA_WARP = 1, EPI_WARP0 = 2;
    const int NST = p.stages, T = p.T;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // same offset in every CTA of the cluster
    uint8_t *smem = smem_raw + (base - raw);
    const uint32_t x_stage = uint32_t(lin::KPS * T) * 128u;
    const uint32_t sW = base;
    const uint32_t sX = base + uint32_t(NST) * lin::W_STAGE_BYTES;
    const uint32_t ring = uint32_t(NST) * (lin::W_STAGE_BYTES + x_stage);
    const uint32_t bar0 = base + ring;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (lin::SPLIT_MAX_STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * lin::SPLIT_MAX_STAGES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + ring + lin::SPLIT_BARS * 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int S = p.split;
    const uint32_t rank = S > 1 ? cluster_ctarank() : 0u;
    // rows of C vary fastest, so that the CTAs sharing weights run together
    const int32_t tile = int32_t(blockIdx.x) / S;
    const int32_t tn = tile / p.sched.nm, tm = tile - tn * p.sched.nm;
    const int32_t m0 = tm * T, n0 = tn * lin::SPLIT_ROWS;
    // this CTA's stages: of the pairs of k-blocks (a last odd one is completed with zeros)
    const int32_t steps = (p.num_kb + lin::KPS - 1) / lin::KPS;
    const int32_t st0 = int32_t(int64_t(steps) * rank / S), st1 = int32_t(int64_t(steps) * (rank + 1) / S);
    const int valid = int(p.M - m0 < T ? p.M - m0 : T);  // rows of C in this tile

    bool ready = false;  // epilogue warps: the accumulator is complete
    uint32_t tmem_base = 0;
    const int ew = warp - EPI_WARP0;
    const bool vec = p.e.vec4 && int64_t(n0) + lin::SPLIT_ROWS <= p.N;  // n0 may lie within 128 of 2^31
    SplitColumns columns = {};

    const uint32_t w_piece = p.b.mn ? lin::KPS * MN_CHUNK_BYTES : lin::SPLIT_ROWS * 128;  // between an operand's copies
    const uint32_t x_piece = p.a.mn ? lin::KPS * MN_CHUNK_BYTES : uint32_t(T) * 128u;
    auto load_w = [&](auto mode, auto mn, int32_t st, uint32_t stage) {
        issue_copies<decltype(mode)::value, decltype(mn)::value, false>(&tmW, sW + stage * lin::W_STAGE_BYTES, w_piece, p.b.copies,
                                                                        st * lin::KPS, BKE, n0, full_bar(stage), lane);
    };
    auto load_x = [&](auto mode, auto mn, int32_t st, uint32_t stage) {
        issue_copies<decltype(mode)::value, decltype(mn)::value, false>(&tmX, sX + stage * x_stage, x_piece, p.a.copies,
                                                                        st * lin::KPS, BKE, m0, full_bar(stage), lane);
    };
    // The stages after the first NST, each once the MMAs have freed its place. After
    // a wait ran out, copies already issued get time to land before the CTA ends.
    auto later_stages = [&](auto load) {
        uint32_t stage = 0, phase = 0;
        for (int32_t st = st0 + NST; st < st1; ++st) {
            if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase, p.wait))) {
                let_copies_land();
                break;
            }
            load(st, stage);
            if (++stage == uint32_t(NST)) { stage = 0; phase ^= 1u; }
        }
        __syncwarp();
    };

    if (warp == 0) {
        // ============================================================ producer (weights)
        // This warp sets up the barriers and starts the first stages by itself, while
        // the others set up tensor memory; only then it meets them.
        if (lane == 0) {
            prefetch_tensormap(&tmW);
            prefetch_tensormap(&tmX);
            for (int s = 0; s < NST; ++s) {
                mbar_init(full_bar(s), 1);
                mbar_init(empty_bar(s), 1);
            }
            mbar_init(done_bar, 1);
            fence_mbar_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
        const int32_t first = min(st0 + NST, st1);
        // the first stages' weights are on their way into L2 while the kernel before ends
        with_load(p.b, [&](auto mode, auto mn) {
            for (int32_t st = st0; st < first; ++st)
                prefetch_copies<decltype(mode)::value, decltype(mn)::value>(&tmW, st * lin::KPS, BKE, n0);
        });
        if (!p.late) griddep_wait();
        // the first stages, both operands
        for (int32_t st = st0; st < first; ++st) mbar_expect_tx_elect(full_bar(st - st0), lin::W_STAGE_BYTES + x_stage);
        with_load(p.b, [&](auto mode, auto mn) {
            for (int32_t st = st0; st < first; ++st) load_w(mode, mn, st, uint32_t(st - st0));
        });
        with_load(p.a, [&](auto mode, auto mn) {
            for (int32_t st = st0; st < first; ++st) load_x(mode, mn, st, uint32_t(st - st0));
        });
        __syncthreads();  // the others are set up; tensor memory is allocated
        griddep_launch_dependents();
        with_load(p.b, [&](auto mode, auto mn) {
            later_stages([&](int32_t st, uint32_t stage) {
                mbar_expect_tx_elect(full_bar(stage), lin::W_STAGE_BYTES + x_stage);
                load_w(mode, mn, st, stage);
            });
        });
    } else {
        if (warp == MMA_WARP) {
            tmem_alloc(smem_addr(tmem_slot), uint32_t(p.tmem_cols));
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        griddep_enter(p.late);
        tmem_base = *tmem_slot;
    }

    if (warp == EPI_WARP0) {
        // ============================================================ producer (tokens), then epilogue
        with_load(p.a, [&](auto mode, auto mn) {
            later_stages([&](int32_t st, uint32_t stage) { load_x(mode, mn, st, stage); });
        });
    }
    if (warp == MMA_WARP) {
        // ============================================================ MMA issuer
        uint32_t stage = 0, phase = 0;
        // descriptors of stage 0; a 32-byte step of K-major K is followed by the next
        // k-block's rows after four, of MN-major K by the next 16 rows of its chunk
        auto desc = [](uint32_t at, uint32_t mn) {
            return mn ? smem_desc(at, lin::KPS * MN_CHUNK_BYTES, 1024) : smem_desc(at, 16, 1024);
        };
        const uint64_t dw = desc(sW, p.b.mn), dx = desc(sX, p.a.mn);
        const uint32_t w_k = (p.b.mn ? UMMA_K * 128u : 32u) >> 4, x_k = (p.a.mn ? UMMA_K * 128u : 32u) >> 4;
        const uint32_t w_kb = p.b.mn ? 4u * w_k : (lin::SPLIT_ROWS * 128u) >> 4, x_kb = p.a.mn ? 4u * x_k : (uint32_t(T) * 128u) >> 4;
        const uint32_t idesc = p.idesc;
        for (int32_t st = st0; st < st1; ++st) {
            if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, p.wait))) break;
            tc_fence_after();
            const uint64_t w0 = dw + stage * (lin::W_STAGE_BYTES >> 4);
            const uint64_t x0 = dx + stage * (x_stage >> 4);
#pragma unroll
            for (int ks = 0; ks < 4 * lin::KPS; ++ks) {
                const uint32_t accumulate = st != st0 || ks != 0 ? 1u : 0u;
                const uint64_t wd = w0 + (ks / 4) * w_kb + (ks % 4) * w_k, xd = x0 + (ks / 4) * x_kb + (ks % 4) * x_k;
                if constexpr (kF8) mma_f8_elect(tmem_base, wd, xd, idesc, accumulate);
                else mma_f16_elect(tmem_base, wd, xd, idesc, accumulate);
            }
            mma_commit_elect(empty_bar(stage));
            if (++stage == uint32_t(NST)) { stage = 0; phase ^= 1u; }
        }
        // also what the epilogue waits for; after a wait that ran out, no MMA may
        // still be writing TMEM when it is freed
        mma_commit_elect(done_bar);
        __all_sync(0xffffffffu, mbar_wait_slow(done_bar, 0, cleanup_wait(p.wait), false));
    } else if (warp >= EPI_WARP0) {
        if (vec) split_columns<kScaled, true>(p, S, rank, ew, lane, m0, n0, valid, columns);
        else split_columns<kScaled, false>(p, S, rank, ew, lane, m0, n0, valid, columns);
        ready = __all_sync(0xffffffffu, mbar_wait(done_bar, 0, p.wait));
        tc_fence_after();
    }

    // ---------------------------------------------------------------- the cluster's sum and the epilogue
    // Each CTA sends the rows of its partial tile to the CTAs they belong to, into
    // the place of their rings: those hold nothing any more once every CTA has met
    // the barrier with its accumulator complete. After the next barrier each CTA
    // finds all it has to add in its own shared memory. (Reading the others' rows
    // instead, after one barrier, left each row waiting for the cluster's latency:
    // 1000 x 640 x 256 9.7 us.)
    __syncwarp();
    if (S > 1) cluster_sync();
    else __syncthreads();
    if (ready) {
        // two warps per TMEM lane quarter: rows [0, T/2) and [T/2, T) of the tile
        const int q = warp & 3, t0 = (ew / 4) * (T / 2);
        with_split(S, [&](auto s) {
            split_send<decltype(s)::value>(tmem_base + (uint32_t(q * 32) << 16), base, rank, q * 32 + lane, t0,
                                           min(t0 + T / 2, valid), p.tmem_cols);
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
            if (vec && one) split_rows<kScaled, SPLIT, true, 1>(p, base, rank, ew, lane, m0, n0, valid, columns);
            else if (vec) split_rows<kScaled, SPLIT, true, kSplitRows>(p, base, rank, ew, lane, m0, n0, valid, columns);
            else split_rows<kScaled, SPLIT, false, kSplitRows>(p, base, rank, ew, lane, m0, n0, valid, columns);
        });
    }
    griddep_leave(p.late);
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem_base, uint32_t(p.tmem_cols));
    }
}

// ================================================================== K = 0
// The sum is empty: C = act(bias) + R, a strip of columns per block, whose bias is
// read once, on every gridDim.y-th row (4096 x 8192 fp16: 21.3 us; a case of the
// definition, not of any model).
__global__ void linear_empty_kernel(const LinearParams p) {
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t j = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; j < p.N; j += int64_t(gridDim.x) * blockDim.x) {
        const float x = p.e.bias != nullptr ? load_elem(p.e.bias, p.e.bias_type, j) : 0.0f;
        const float y = act_one(p.e.act, x);
        for (int64_t i = blockIdx.y; i < p.M; i += gridDim.y) {
            if (p.e.pre != nullptr) store_elem(p.e.pre, p.e.type, i * p.e.ldp + j, x);
            store_elem(p.e.c, p.e.type, i * p.e.ldc + j, p.e.r != nullptr ? y + load_elem(p.e.r, p.e.type, i * p.e.ldr + j) : y);
        }
    }
}

// ================================================================== 8-bit operand copies
// Rows of `inner` bytes, any base and pitch -> rows on 128-byte lines (dst 128-byte
// aligned, ld_dst a multiple of 128), zero past `inner`. One 16-byte granule of
// the copy per thread and step, from the one or two aligned source granules that
// hold its bytes (a granule is read only when it holds a byte of the row). Bound by
// latency and DRAM (4096 x 8191 and 128 x 8191: 69 MB moved in about 13 us of the 23.3 of
// a product with them; without copies, at K = 8192, it takes 9.8).
struct PackBytesJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t rows, inner, ld_src, ld_dst;
    int64_t gpr, granules;  // granules per row; rows * gpr, or 0: not copied
};

__global__ void pack_bytes_kernel(PackBytesJob a, PackBytesJob b) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t total = a.granules + b.granules;
    for (int64_t e = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += int64_t(gridDim.x) * blockDim.x) {
        const bool second = e >= a.granules;
        const PackBytesJob &J = second ? b : a;
        const int64_t f = second ? e - a.granules : e;
        const int64_t r = f / J.gpr, i0 = (f - r * J.gpr) * 16;
        if (!G16_CHECK(r < J.rows && i0 < J.inner)) continue;
        const int64_t left = J.inner - i0;
        const uint32_t cnt = left < 16 ? uint32_t(left) : 16u;
        const uintptr_t s = reinterpret_cast<uintptr_t>(J.src + r * J.ld_src + i0);
        const uintptr_t g0 = s & ~uintptr_t(15);
        const uint32_t m = uint32_t(s - g0);
        uint32_t w[9];
        const uint4 lo = *reinterpret_cast<const uint4 *>(g0);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
        uint4 hi = make_uint4(0u, 0u, 0u, 0u);
        if (m + cnt > 16) hi = *reinterpret_cast<const uint4 *>(g0 + 16);
        w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w, w[8] = 0u;
        uint32_t x[7], y[5], o[4];
#pragma unroll
        for (int t = 0; t < 7; ++t) x[t] = (m & 8u) ? w[t + 2] : w[t];
#pragma unroll
        for (int t = 0; t < 5; ++t) y[t] = (m & 4u) ? x[t + 1] : x[t];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            o[t] = __funnelshift_r(y[t], y[t + 1], (m & 3u) * 8u);
            const int keep = int(cnt) - 4 * t;  // bytes of this word inside the row
            if (keep <= 0) o[t] = 0u;
            else if (keep < 4) o[t] &= (1u << (8 * keep)) - 1u;
        }
        *reinterpret_cast<uint4 *>(J.dst + r * J.ld_dst + i0) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ================================================================== backward, elementwise part
// D = G act'(P) and the column sums of D over blocks of rows. A block is 32
// lanes x 8 row groups on a strip of 256 columns (8 per lane); the sums use D
// before its rounding. 4096 x 8192 bf16 with gelu: 201 MB in 38.4 us (5.2 TB/s),
// bound by DRAM and, half of the cycles, by the slope's arithmetic. Without activation
// (the sums alone, 67 MB from DRAM) 22 us with their last step, bound by the loads in
// flight: 512 threads on an SM (122 registers, for the activations) with four each, and
// an end that the last step's launch waits for. Rows off 16-byte boundaries are put
// together from the two granules that hold eight elements (kShift): the sums of 4096 x
// 8191 with gelu 51.0 us, element by element 76.2, on boundaries 36.7.
// D is rounded to G's type because the products that read it run on 16-bit tensor
// cores; as two 16-bit parts it would double their time. Against 64 bits, bf16
// gradients are off by 0.0024 of their norm with it and by 0.0017, their own rounding,
// without.
struct GradParams {
    const void *g, *pre;  // pre == nullptr: D = G
    void *d;              // nullptr: not stored
    float *partial;       // [gridDim.y][N] or nullptr
    int64_t M, N, ldg, ldp, ldd;
    int64_t rows_per_block;
    uint32_t act, late;
};
constexpr int kGradGroups = 8;

// Eight elements of a row from `at` on as they come: the one or, kShift, two
// granules that hold them. They come from L2: with `late` the kernel reads before its
// own wait, what the call's first kernel found complete, and so relies on no L1 line
// that an earlier launch has left.
template <typename T, bool kShift>
struct GradLoad {
    Raw<T, 8> lo, hi;
    __device__ __forceinline__ void fetch(const T *row, int64_t at, int64_t n) {
        if constexpr (kShift) {
            const int s = place_in_granule(row + at);
            lo = load_raw_l2<T>(row + at - s);
            hi.q[0] = make_uint4(0u, 0u, 0u, 0u);
            if (s != 0 && at + 8 - s < n) hi = load_raw_l2<T>(row + at - s + 8);  // only where the row reaches into it
        } else {
            lo = load_raw_l2<T>(row + at);
        }
    }
    // the values, zero from column n on
    __device__ __forceinline__ F32<8> values(const T *row, int64_t at, int64_t n) const {
        if constexpr (kShift) {
            Raw<T, 8> r = shift_granules<T>(lo, hi, place_in_granule(row + at));
            if (at + 8 > n) keep_elems<T>(r, 0, int(n - at));
            return widen<T, 8>(r);
        } else {
            return widen<T, 8>(lo);
        }
    }
};

template <uint32_t ACT, typename T, bool kShift>
__device__ __forceinline__ void grad_rows(const GradParams &p, int64_t col, int64_t r0, int64_t r1, F32<8> &sum) {
    const T *g = static_cast<const T *>(p.g), *pre = static_cast<const T *>(p.pre);
    T *d = static_cast<T *>(p.d);
    constexpr int AHEAD = kShift ? 2 : 4;  // rows loaded before the first is stored
#pragma unroll 1
    for (int64_t r = r0 + threadIdx.y; r < r1; r += AHEAD * kGradGroups) {
        GradLoad<T, kShift> a[AHEAD], b[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * kGradGroups;
            if (row >= r1) break;
            a[k].fetch(g + row * p.ldg, col, p.N);
            if constexpr (ACT != kActNone) b[k].fetch(pre + row * p.ldp, col, p.N);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t row = r + k * kGradGroups;
            if (row >= r1) break;
            F32<8> x = a[k].values(g + row * p.ldg, col, p.N);
            if constexpr (ACT != kActNone) {
                const F32<8> f = b[k].values(pre + row * p.ldp, col, p.N);
#pragma unroll
                for (int i = 0; i < F32<8>::PAIRS; ++i) x.p[i] = mul2(x.p[i], act_slope<ACT>(f.p[i]));
            }
            if (d != nullptr) {
                if constexpr (kShift) store_some<T>(d + row * p.ldd + col, x, 0, int(p.N - col < 8 ? p.N - col : 8));
                else store_f32<T, 8>(d + row * p.ldd + col, x);
            }
#pragma unroll
            for (int i = 0; i < F32<8>::PAIRS; ++i) sum.p[i] = add2(sum.p[i], x.p[i]);
        }
    }
}

// kShift: G's or pre's rows off 16-byte boundaries, or N no multiple of 8.
template <typename T, bool kShift>
__global__ void __launch_bounds__(32 * kGradGroups) linear_grad_kernel(const GradParams p) {
    __shared__ float s[kGradGroups][32 * 8 + 1];
    griddep_enter(p.late);
    const int64_t col = (int64_t(blockIdx.x) * 32 + threadIdx.x) * 8;
    const int64_t r0 = int64_t(blockIdx.y) * p.rows_per_block;
    const int64_t r1 = r0 + p.rows_per_block < p.M ? r0 + p.rows_per_block : p.M;
    F32<8> sum;
#pragma unroll
    for (int i = 0; i < F32<8>::PAIRS; ++i) sum.p[i] = splat<8>(0.0f);
    if (col < p.N) {
        switch (p.act) {
            case kActRelu: grad_rows<kActRelu, T, kShift>(p, col, r0, r1, sum); break;
            case kActGelu: grad_rows<kActGelu, T, kShift>(p, col, r0, r1, sum); break;
            case kActGeluTanh: grad_rows<kActGeluTanh, T, kShift>(p, col, r0, r1, sum); break;
            case kActSilu: grad_rows<kActSilu, T, kShift>(p, col, r0, r1, sum); break;
            default: grad_rows<kActNone, T, kShift>(p, col, r0, r1, sum); break;
        }
    }
    griddep_leave(p.late);
    if (p.partial == nullptr) return;
#pragma unroll
    for (int i = 0; i < F32<8>::PAIRS; ++i) {
        s[threadIdx.y][threadIdx.x * 8 + 2 * i] = sum.p[i].x;
        s[threadIdx.y][threadIdx.x * 8 + 2 * i + 1] = sum.p[i].y;
    }
    __syncthreads();
    for (int c = threadIdx.y * 32 + threadIdx.x; c < 32 * 8; c += 32 * kGradGroups) {
        const int64_t at = int64_t(blockIdx.x) * 32 * 8 + c;
        if (at >= p.N) continue;
        float v = s[0][c];
        for (int y = 1; y < kGradGroups; ++y) v += s[y][c];
        p.partial[int64_t(blockIdx.y) * p.N + at] = v;
    }
}

}  // namespace g16
