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
#include "elements.cuh"
#include "gemm_kernel.cuh"

namespace g16 {

// ------------------------------------------------------------------ launches that overlap
// A kernel of a call that needs nothing of the kernel right before it (late != 0)
// does not wait for it before its work but before it ends. What it does read was
// written by kernels that had completed before that one's own wait returned, and
// so before this one could be scheduled; it comes from L2, by TMA or by loads that
// pass L1. Whatever follows on the stream still finds both complete. In gradients the
// second product's tiles so fill the SMs that the first one's last round leaves idle.
__device__ __forceinline__ void griddep_enter(uint32_t late) {
    if (!late) griddep_wait();
    griddep_launch_dependents();
}
__device__ __forceinline__ void griddep_leave(uint32_t late) {
    if (late) griddep_wait();
}

// ------------------------------------------------------------------ loads past L1 and from shared memory
// Eight elements from L2, past this SM's L1.
template <typename T>
__device__ __forceinline__ Raw<T, 8> load_raw_l2(const T *p) {
    Raw<T, 8> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(r) / 16); ++i) r.q[i] = __ldcg(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}

// The same from a shared-memory address (VEC = 8: 16-byte aligned).
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw_shared(uint32_t addr) {
    Raw<T, VEC> r;
    if constexpr (VEC == 8) {
#pragma unroll
        for (int i = 0; i < int(sizeof(r) / 16); ++i) ld_shared_v4(addr + 16u * i, r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w);
    } else if constexpr (sizeof(T) == 4) {
        const uint32_t w = ld_shared_b32(addr);
        r.v = *reinterpret_cast<const T *>(&w);
    } else {
        uint16_t w = 0;
        if (G16_CHECK(smem_window_ok(addr, 2))) asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(addr) : "memory");
        r.v = *reinterpret_cast<const T *>(&w);
    }
    return r;
}

constexpr float kQuantTwoSteps = 1.4e-36f;  // below this, 448 / x may leave fp32's range

// With t = w h, y = t rstd and a = max|y| = rstd max|t|, so y 448 / a = t 448 /
// max|t|: the row's factor `mul` for t and its scale, from max|t|. One pass over the
// row then gives both its sum and its maximum. Where max|t| is too small for that
// quotient while a is not, t is first multiplied by rstd (`first`, else 1), then by
// 448 / a. An infinity or a NaN among y makes the row and its scale NaN. (max|t| = 0
// is looked at by itself: without eps, a zero row's rstd is infinite.)
__device__ __forceinline__ void quant_factors(float tmax, float rstd, float &first, float &mul, float &scale) {
    const float a = tmax * rstd;
    first = 1.0f;
    if (tmax == 0.0f || a < kQuantTiny) {
        mul = 0.0f;
        scale = 1.0f;
    } else if (!(a <= kLargest)) {
        mul = scale = __int_as_float(0x7fffffff);  // NaN
    } else {
        if (tmax < kQuantTwoSteps) {
            first = rstd;
            mul = kE4m3Max / a;
        } else {
            mul = kE4m3Max / tmax;
        }
        scale = a * (1.0f / kE4m3Max);
    }
}

// t = w h of VEC elements; adds h^2 to ss and takes |t| into tmax.
template <int VEC, bool kQ>
__device__ __forceinline__ void square_and_weigh(F32<VEC> &t, const F32<VEC> &w, typename F32<VEC>::E &ss, float &tmax) {
#pragma unroll
    for (int i = 0; i < F32<VEC>::PAIRS; ++i) {
        ss = fma2(t.p[i], t.p[i], ss);
        t.p[i] = mul2(t.p[i], w.p[i]);
        if constexpr (kQ && VEC == 8) tmax = max_nan(max_nan(tmax, fabsf(t.p[i].x)), fabsf(t.p[i].y));
        else if constexpr (kQ) tmax = max_nan(tmax, fabsf(t.p[i]));
    }
}

struct NormParams {
    const void *x, *r;  // r == nullptr: no residual
    const void *w;
    void *y, *h;  // h == nullptr: not stored
    float *scale, *rstd;
    int64_t rows, width;
    int64_t ldx, ldr, ldy, ldh;
    float eps, inv_width;
    int32_t w_f32;
    WaitCtl wait;
};

// One row per blockDim.x threads, held in registers: element (j * blockDim.x +
// t) * VEC + i of the row is value i of load j of thread t.
// kShift: rows off 16-byte boundaries, their first element `o` into a granule.
// DRAM bounds it where there are many rows (8192 x 4096 bf16 with residual: 268 MB
// in 41 us, 6.5 TB/s; 4096 x 8192 to 8 bits 235 MB in 36.9 us, 6.4 TB/s), the chain
// load - reduction - store where there are few (1 x 4096: 2.0 us).
template <typename T, int VEC, int NV, bool kQ, bool kShift>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
    __shared__ float red[32];
    __shared__ uint32_t redq[32];
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    griddep_wait();
    griddep_launch_dependents();
    const int width = int(p.width);
    const int o = kShift && live ? place_in_granule(static_cast<const T *>(p.x) + row * p.ldx) : 0;
    auto at_of = [&](int j) { return (j * int(blockDim.x) + int(threadIdx.x)) * VEC - o; };
    F32<VEC> t[NV];
    {
        Raw<T, VEC> a[NV], b[NV];
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *r = static_cast<const T *>(p.r) + row * p.ldr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!live || at_of(j) >= width) continue;
            a[j] = load_raw<T, VEC>(x + at_of(j));
            if (p.r != nullptr) b[j] = load_raw<T, VEC>(r + at_of(j));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!live || at_of(j) >= width) continue;
            if constexpr (kShift) {
                if (at_of(j) < 0 || at_of(j) + VEC > width) {
                    keep_elems<T>(a[j], -at_of(j), width - at_of(j));
                    if (p.r != nullptr) keep_elems<T>(b[j], -at_of(j), width - at_of(j));
                }
            }
            t[j] = widen<T, VEC>(a[j]);
            if (p.r == nullptr) continue;
            const F32<VEC> f = widen<T, VEC>(b[j]);
#pragma unroll
            for (int i = 0; i < F32<VEC>::PAIRS; ++i) t[j].p[i] = add2(t[j].p[i], f.p[i]);
        }
    }
    auto ss2 = splat<VEC>(0.0f);
    float tmax = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!live || at_of(j) >= width) continue;
        if constexpr (kShift) {
            if (p.h != nullptr)
                store_some<T>(static_cast<T *>(p.h) + row * p.ldh + at_of(j), t[j], -at_of(j), width - at_of(j));
            square_and_weigh<VEC, kQ>(t[j], widen<T, VEC>(load_shifted<T>(static_cast<const T *>(p.w), at_of(j), width)), ss2, tmax);
        } else {
            if (p.h != nullptr) store_f32<T, VEC>(static_cast<T *>(p.h) + row * p.ldh + at_of(j), t[j]);
            square_and_weigh<VEC, kQ>(t[j], load_weight<T, VEC>(p.w, p.w_f32 != 0, at_of(j)), ss2, tmax);
        }
    }
    float ss = total(ss2);
    if constexpr (kQ) row_sum_max(ss, tmax, red, redq);
    else ss = row_sum<false>(ss, red);
    const float rstd = rsqrtf(fmaf(ss, p.inv_width, p.eps));
    if (!live) return;
    if (p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
    float mul = rstd;
    if constexpr (kQ) {
        float scale, first;
        quant_factors(tmax, rstd, first, mul, scale);
        if (threadIdx.x == 0) p.scale[row] = scale;
        if (first != 1.0f) {  // the whole row; rare
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (at_of(j) >= width) continue;
#pragma unroll
                for (int i = 0; i < F32<VEC>::PAIRS; ++i) t[j].p[i] = mul2(t[j].p[i], splat<VEC>(first));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (at_of(j) >= width) continue;
#pragma unroll
        for (int i = 0; i < F32<VEC>::PAIRS; ++i) t[j].p[i] = mul2(t[j].p[i], splat<VEC>(mul));
        if constexpr (kShift)
            store_some<std::conditional_t<kQ, uint8_t, T>>(static_cast<std::conditional_t<kQ, uint8_t, T> *>(p.y) + row * p.ldy + at_of(j),
                                                           t[j], -at_of(j), width - at_of(j));
        else if constexpr (kQ) store_e4m3<VEC>(static_cast<uint8_t *>(p.y) + row * p.ldy + at_of(j), t[j]);
        else store_f32<T, VEC>(static_cast<T *>(p.y) + row * p.ldy + at_of(j), t[j]);
    }
}

// Rows longer than the register form holds: one block per row, which reads its
// row once per pass (sum and, with 8 bits, the maximum; store) element by element; a
// thread re-reads only what it wrote itself, so h may be x or r. The second pass finds
// the row in L2 (512 x 40000 bf16 with residual: 55.9 us for 164 MB, 2.9 TB/s,
// bound by instructions per element).
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
    float ss = 0.0f, tmax = 0.0f;
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float h = sum(at);
        ss = fmaf(h, h, ss);
        if (quant) tmax = max_nan(tmax, fabsf(h * load_weight<T, 1>(p.w, p.w_f32 != 0, at).p[0]));
    }
    row_sum_max(ss, tmax, red, redq);
    const float rstd = rsqrtf(fmaf(ss, p.inv_width, p.eps));
    if (p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
    float mul = rstd, first = 1.0f, scale = 1.0f;
    if (quant) {
        quant_factors(tmax, rstd, first, mul, scale);
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float h = sum(at);
        F32<1> y;
        y.p[0] = h * load_weight<T, 1>(p.w, p.w_f32 != 0, at).p[0] * first * mul;
        if (p.h != nullptr) static_cast<T *>(p.h)[row * p.ldh + at] = from_f32<T>(h);
        if (quant) store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.ldy + at, y);
        else store_f32<T, 1>(static_cast<T *>(p.y) + row * p.ldy + at, y);
    }
}

// ------------------------------------------------------------------ rows through shared memory
// The persistent form: each block walks rows base + threadIdx.y, base = blockIdx.x
// * blockDim.y, then every gridDim.x * blockDim.y further on. The rows of the next
// steps are on their way into a ring of shared-memory slots (bulk copies) while
// this one is summed and written, so the memory system stays busy through the
// barriers of the reductions. A copy starts and ends on 16-byte boundaries: it
// takes the bytes that share a granule with the row's first and last element
// too, and the row's elements are found from the offset in that granule.
constexpr int kRingSlots = 8;      // at most
constexpr int kRingThreads = 512;  // at most: 128 registers each, so two blocks of 256 share an SM

struct RingShape {
    int32_t slots;
    int32_t pitch;        // bytes between the rows of one array in a slot
    int32_t array_bytes;  // rows of a slot * pitch
    int32_t slot_bytes;   // arrays * array_bytes
};

template <typename T>
struct RowSource {
    const T *data;
    int64_t ld;
    __device__ __forceinline__ uint32_t in_slot(uint32_t place, int64_t row) const {
        return place + (uint32_t(reinterpret_cast<uintptr_t>(data + row * ld)) & 15u);
    }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    if (!G16_CHECK((bytes & 15u) == 0 && smem_window_ok(dst, bytes))) return;
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// Warp 0 of the block starts the copies of a slot's rows of every array, one lane
// per copy: rows base .. base + nrows - 1 or, where R rows of a thread are `apart`
// rows from each other, row q of the slot is base + q / R + (q mod R) apart.
template <typename T, int R = 1>
__device__ __forceinline__ void fill_slot(const RowSource<T> *src, int arrays, int nrows, const RingShape &ring, uint8_t *slots,
                                          int slot, uint32_t bar, int64_t base, int64_t rows, int64_t width, int64_t apart = 1) {
    if (threadIdx.y != 0 || threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    const int a = lane / nrows, y = lane - a * nrows;
    const int64_t row = apart == 1 ? base + y : base + y / R + (y % R) * apart;
    uint32_t bytes = 0, dst = 0;
    const void *from = nullptr;
    if (a < arrays && row < rows) {
        const RowSource<T> s = a == 0 ? src[0] : a == 1 ? src[1] : src[2];
        const uintptr_t at = reinterpret_cast<uintptr_t>(s.data + row * s.ld);
        from = reinterpret_cast<const void *>(at & ~uintptr_t(15));
        bytes = (uint32_t(at & 15u) + uint32_t(width) * uint32_t(sizeof(T)) + 15u) & ~15u;
        dst = smem_addr(slots) + uint32_t(slot * ring.slot_bytes + a * ring.array_bytes + y * ring.pitch);
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (bytes > 0) bulk_load(dst, from, bytes, bar);
}

// After a wait ran out (the status is set, the results are not to be used): time
// for copies already started, rows of some 64 KiB at most, to land before the
// block's shared memory is given away.
__device__ __forceinline__ void let_copies_land() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000ull) {
    }
}

// Rows that neither lie on 16-byte boundaries nor all start at the same place in
// a granule, or fp32 ones off them: element by element out of the slots, lane by
// lane along the row, so that the stores of a warp stay contiguous. A slot is read
// twice and refilled after the next step's barrier. Bound by instructions (4096 x
// 4095 fp16 with residual, y one element further on: 66.4 us, where the same place
// takes 26.5; fp32 71.2, 4096 x 4096 42.2).
template <typename T>
__device__ __forceinline__ float lds_elem(uint32_t row, int c) {
    return to_f32<T>(load_raw_shared<T, 1>(row + uint32_t(c) * uint32_t(sizeof(T))).v);
}

template <typename T, bool kQ>
__global__ void __launch_bounds__(kRingThreads) rms_norm_rows_any_kernel(const NormParams p, const RingShape ring) {
    __shared__ float red[2][32];
    __shared__ uint32_t redq[2][32];
    __shared__ __align__(8) uint64_t full[kRingSlots];
    extern __shared__ __align__(16) uint8_t rows[];
    if (threadIdx.y == 0 && threadIdx.x == 0) {
        for (int s = 0; s < ring.slots; ++s) mbar_init(smem_addr(&full[s]), 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y;
    const RowSource<T> src[3] = {{static_cast<const T *>(p.x), p.ldx}, {static_cast<const T *>(p.r), p.ldr}, {nullptr, 0}};
    const bool has_r = p.r != nullptr, has_h = p.h != nullptr;
    auto refill = [&](int64_t base, int slot) {
        if (base < p.rows) fill_slot(src, has_r ? 2 : 1, int(blockDim.y), ring, rows, slot, smem_addr(&full[slot]), base, p.rows, p.width);
    };
    for (int s = 0; s < ring.slots; ++s) refill(first + s * step, s);
    const int width = int(p.width), tpr = int(blockDim.x);
    const uint32_t ring0 = smem_addr(rows) + uint32_t(int(threadIdx.y) * ring.pitch);
    int slot = 0, last = ring.slots - 1, flip = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t base = first; base < p.rows; base += step, flip ^= 1) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < p.rows;
        ok = mbar_wait(smem_addr(&full[slot]), phase, p.wait) && ok;
        const uint32_t mine = ring0 + uint32_t(slot * ring.slot_bytes);
        const uint32_t x = src[0].in_slot(mine, row), r = src[1].in_slot(mine + uint32_t(ring.array_bytes), row);
        auto sum = [&](int c) { return lds_elem<T>(x, c) + (has_r ? lds_elem<T>(r, c) : 0.0f); };
        float ss = 0.0f, tmax = 0.0f;
        if (live) {
#pragma unroll 4
            for (int c = threadIdx.x; c < width; c += tpr) {
                const float h = sum(c);
                ss = fmaf(h, h, ss);
                if (kQ) tmax = max_nan(tmax, fabsf(h * load_weight<T, 1>(p.w, p.w_f32 != 0, c).p[0]));
            }
        }
        if constexpr (kQ) row_sum_max(ss, tmax, red[flip], redq[flip]);
        else ss = row_sum<true>(ss, red[flip]);
        if (base >= first + step) refill(base + int64_t(ring.slots - 1) * step, last);  // all have left the step before
        const float rstd = rsqrtf(fmaf(ss, p.inv_width, p.eps));
        float mul = rstd, first = 1.0f;
        if constexpr (kQ) {
            float scale;
            quant_factors(tmax, rstd, first, mul, scale);
            if (live && threadIdx.x == 0) p.scale[row] = scale;
        }
        if (live && p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
        if (live) {
            T *ho = static_cast<T *>(p.h) + row * p.ldh;
#pragma unroll 4
            for (int c = threadIdx.x; c < width; c += tpr) {
                const float h = sum(c);
                if (has_h) ho[c] = from_f32<T>(h);
                F32<1> y;
                y.p[0] = h * load_weight<T, 1>(p.w, p.w_f32 != 0, c).p[0];
                if constexpr (kQ) y.p[0] *= first;
                y.p[0] *= mul;
                if constexpr (kQ) store_e4m3<1>(static_cast<uint8_t *>(p.y) + row * p.ldy + c, y);
                else store_f32<T, 1>(static_cast<T *>(p.y) + row * p.ldy + c, y);
            }
        }
        last = slot;
        if (++slot == ring.slots) { slot = 0; phase ^= 1u; }
    }
    if (!ok) let_copies_land();
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
    WaitCtl wait;
};

// The persistent form: rows arrive through a ring of shared-memory slots, and a
// thread keeps its columns, so that their dweight sums stay in its registers and
// each block writes one row of partial sums at its end. A slot is read twice (for the row's dot product and for dx) and
// refilled after the next step's barrier. The chain of a row's reduction is long
// beside its arithmetic, so a thread works on R rows at a time (row base +
// threadIdx.y * R + r), with one barrier for all of them. 8192 x 4096 bf16 with
// grad_h: 268 MB in 50.1 us with the sum of the partials, 45 of them here: 6.0 TB/s,
// bound by DRAM; half of the issue slots are busy.
// kShift: rows off 16-byte boundaries. A thread's rows are then a multiple of 8
// rows apart (its block's next ones, the grid being a multiple of 8), so that all of
// them start at the same place in a granule and a thread keeps its columns.
template <typename T, int NV, int R, bool kShift>
__global__ void __launch_bounds__(kRingThreads) rms_norm_backward_rows_kernel(const NormBackwardParams p, const RingShape ring) {
    constexpr int VEC = 8;
    __shared__ float red[2][R][32];
    __shared__ __align__(8) uint64_t full[kRingSlots];
    extern __shared__ __align__(16) uint8_t rows[];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    if (tid == 0) {
        for (int s = 0; s < ring.slots; ++s) mbar_init(smem_addr(&full[s]), 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int per_slot = int(blockDim.y) * R;
    const int64_t step = int64_t(gridDim.x) * per_slot;
    const int64_t first = int64_t(blockIdx.x) * (kShift ? int(blockDim.y) : per_slot);
    const int64_t apart = kShift && R > 1 ? int64_t(gridDim.x) * blockDim.y : 1;  // rows between a thread's R rows
    const RowSource<T> src[3] = {{static_cast<const T *>(p.g), p.ldg}, {static_cast<const T *>(p.h), p.ldh},
                                 {static_cast<const T *>(p.dh), p.lddh}};
    const bool has_d = p.dh != nullptr;
    auto refill = [&](int64_t base, int slot) {
        if (base < p.rows)
            fill_slot<T, R>(src, has_d ? 3 : 2, per_slot, ring, rows, slot, smem_addr(&full[slot]), base, p.rows, p.width, apart);
    };
    for (int s = 0; s < ring.slots; ++s) refill(first + s * step, s);
    int64_t row = first + int64_t(threadIdx.y) * (kShift ? 1 : R);
    const int o = kShift && row < p.rows ? place_in_granule(static_cast<const T *>(p.g) + row * p.ldg) : 0;
    auto at_of = [&](int j) { return (j * int(blockDim.x) + int(threadIdx.x)) * VEC - o; };
    const int width = int(p.width);
    auto cut = [&](int j) { return kShift && (at_of(j) < 0 || at_of(j) + VEC > width); };
    F32<VEC> dw[NV];
    Raw<T, VEC> w16[NV];  // a weight of T's type; fp32 weights are read again for each row
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < F32<VEC>::PAIRS; ++i) dw[j].p[i] = splat<VEC>(0.0f);
        if (at_of(j) >= width || p.w_f32) continue;
        if constexpr (kShift) w16[j] = load_shifted<T>(static_cast<const T *>(p.w), at_of(j), width);
        else w16[j] = load_raw<T, VEC>(static_cast<const T *>(p.w) + at_of(j));
    }
    auto weight = [&](int j) { return !kShift && p.w_f32 ? load_weight<T, VEC>(p.w, true, at_of(j)) : widen<T, VEC>(w16[j]); };
    const uint32_t ring0 = smem_addr(rows) + uint32_t(int(threadIdx.y) * R * ring.pitch);
    const uint32_t off_h = uint32_t(ring.array_bytes), off_d = 2u * off_h;
    int slot = 0, last = ring.slots - 1;  // `last`: the slot before it in the ring
    uint32_t phase = 0;
    int flip = 0;
    bool ok = true;
    T *dx = static_cast<T *>(p.dx) + row * p.lddx;
    const int64_t dx_step = step * p.lddx;
    float rs_next[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rs_next[r] = row + r * apart < p.rows ? p.rstd[row + r * apart] : 0.0f;
    for (int64_t base = first; base < p.rows; base += step, row += step, dx += dx_step, flip ^= 1) {
        float rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rs[r] = rs_next[r];
            rs_next[r] = row + step + r * apart < p.rows ? p.rstd[row + step + r * apart] : 0.0f;
        }
        ok = mbar_wait(smem_addr(&full[slot]), phase, p.wait) && ok;
        const uint32_t mine = ring0 + uint32_t(slot * ring.slot_bytes);
        int left = 0;  // rows of this thread that exist
#pragma unroll
        for (int r = 0; r < R; ++r) left += row + r * apart < p.rows;
        Raw<T, VEC> rg[R][NV], rh[R][NV];
        float sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t g = mine + uint32_t(r * ring.pitch);
            auto dot2 = splat<VEC>(0.0f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (r >= left || at_of(j) >= width) continue;
                const uint32_t at = g + uint32_t(at_of(j) + o) * uint32_t(sizeof(T));
                rg[r][j] = load_raw_shared<T, VEC>(at);
                rh[r][j] = load_raw_shared<T, VEC>(at + off_h);
                if constexpr (kShift) {
                    if (cut(j)) {
                        keep_elems<T>(rg[r][j], -at_of(j), width - at_of(j));
                        keep_elems<T>(rh[r][j], -at_of(j), width - at_of(j));
                    }
                }
                const F32<VEC> fg = widen<T, VEC>(rg[r][j]), fh = widen<T, VEC>(rh[r][j]), w = weight(j);
#pragma unroll
                for (int i = 0; i < F32<VEC>::PAIRS; ++i) dot2 = fma2(mul2(fg.p[i], w.p[i]), fh.p[i], dot2);
            }
            sum[r] = total(dot2);
        }
        rows_sum<R>(sum, red[flip]);
        if (base >= first + step) refill(base + int64_t(ring.slots - 1) * step, last);  // all have left the step before
        // dx = rstd g + (-rstd mean(g u)) u + dh, with g = dy w, u = h rstd
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const auto rs2 = splat<VEC>(rs[r]), c2 = splat<VEC>(-rs[r] * (sum[r] * rs[r] * p.inv_width));
            const uint32_t d = mine + uint32_t(r * ring.pitch) + off_d;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (r >= left || at_of(j) >= width) continue;
                const F32<VEC> fg = widen<T, VEC>(rg[r][j]), fh = widen<T, VEC>(rh[r][j]), w = weight(j);
                F32<VEC> v;
                if (has_d) v = widen<T, VEC>(load_raw_shared<T, VEC>(d + uint32_t(at_of(j) + o) * uint32_t(sizeof(T))));
#pragma unroll
                for (int i = 0; i < F32<VEC>::PAIRS; ++i) {
                    const auto u = mul2(fh.p[i], rs2);
                    dw[j].p[i] = fma2(fg.p[i], u, dw[j].p[i]);
                    const auto gw = mul2(fg.p[i], w.p[i]);
                    v.p[i] = fma2(u, c2, has_d ? fma2(gw, rs2, v.p[i]) : mul2(gw, rs2));
                }
                T *to = dx + r * apart * p.lddx + at_of(j);
                if constexpr (kShift) store_some<T>(to, v, -at_of(j), width - at_of(j));
                else store_f32<T, VEC>(to, v);
            }
        }
        last = slot;
        if (++slot == ring.slots) { slot = 0; phase ^= 1u; }
    }
    if (!ok) let_copies_land();
    if (p.partial == nullptr) return;
    float *out = p.partial + int64_t(blockIdx.x) * p.width;
    if (kShift || blockDim.y > 1) {
        // through shared memory (the ring holds no copy in flight any more): the block's
        // rows added up in order, and stores that are contiguous over a warp
        float *dw_rows = reinterpret_cast<float *>(rows);
        const int span = blockDim.x * VEC * NV;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (kShift) store_elems(dw_rows + int(threadIdx.y) * span + at_of(j), dw[j], -at_of(j), width - at_of(j));
            else store_f32<float, VEC>(dw_rows + int(threadIdx.y) * span + at_of(j), dw[j]);
        }
        __syncthreads();
        for (int c = tid; c < span && c < width; c += blockDim.x * blockDim.y) {
            float s = dw_rows[c];
            for (int y = 1; y < int(blockDim.y); ++y) s += dw_rows[y * span + c];
            out[c] = s;
        }
        return;
    }
    if constexpr (!kShift) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (at_of(j) >= width) continue;
            store_f32<float, VEC>(out + at_of(j), dw[j]);  // width is a multiple of 8, the workspace aligned
        }
    }
}

// Any alignment and width, as rms_norm_rows_any_kernel; the dweight sums are in
// shared memory behind the ring, one row of them per row of the block, each
// column touched by its own thread only. Bound by instructions (4096 x 4095 fp16
// with grad_h, dx one element further on: 69.8 us, where the same place takes 39.2).
template <typename T>
__global__ void __launch_bounds__(kRingThreads) rms_norm_backward_rows_any_kernel(const NormBackwardParams p, const RingShape ring) {
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t full[kRingSlots];
    extern __shared__ __align__(16) uint8_t rows[];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, width = int(p.width), tpr = int(blockDim.x);
    float *dw_rows = reinterpret_cast<float *>(rows + ring.slots * ring.slot_bytes);
    float *dw = dw_rows + int(threadIdx.y) * width;
    if (tid == 0) {
        for (int s = 0; s < ring.slots; ++s) mbar_init(smem_addr(&full[s]), 1);
        fence_mbar_init();
    }
    for (int c = threadIdx.x; c < width; c += tpr) dw[c] = 0.0f;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y;
    const RowSource<T> src[3] = {{static_cast<const T *>(p.g), p.ldg}, {static_cast<const T *>(p.h), p.ldh},
                                 {static_cast<const T *>(p.dh), p.lddh}};
    const bool has_d = p.dh != nullptr;
    auto refill = [&](int64_t base, int slot) {
        if (base < p.rows) fill_slot(src, has_d ? 3 : 2, int(blockDim.y), ring, rows, slot, smem_addr(&full[slot]), base, p.rows, p.width);
    };
    for (int s = 0; s < ring.slots; ++s) refill(first + s * step, s);
    const uint32_t ring0 = smem_addr(rows) + uint32_t(int(threadIdx.y) * ring.pitch);
    int slot = 0, last = ring.slots - 1, flip = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto rstd_of = [&](int64_t row) { return row < p.rows ? p.rstd[row] : 0.0f; };
    float rs_next = rstd_of(first + threadIdx.y);
    for (int64_t base = first; base < p.rows; base += step, flip ^= 1) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < p.rows;
        const float rs = rs_next;
        rs_next = rstd_of(row + step);
        ok = mbar_wait(smem_addr(&full[slot]), phase, p.wait) && ok;
        const uint32_t mine = ring0 + uint32_t(slot * ring.slot_bytes);
        const uint32_t g = src[0].in_slot(mine, row), h = src[1].in_slot(mine + uint32_t(ring.array_bytes), row),
                       d = src[2].in_slot(mine + 2u * uint32_t(ring.array_bytes), row);
        float dot = 0.0f;
        if (live) {
#pragma unroll 4
            for (int c = threadIdx.x; c < width; c += tpr)
                dot = fmaf(lds_elem<T>(g, c) * load_weight<T, 1>(p.w, p.w_f32 != 0, c).p[0], lds_elem<T>(h, c), dot);
        }
        const float sum = row_sum<true>(dot, red[flip]);
        if (base >= first + step) refill(base + int64_t(ring.slots - 1) * step, last);  // all have left the step before
        if (live) {
            const float m = -rs * (sum * rs * p.inv_width);
            T *dx = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll 4
            for (int c = threadIdx.x; c < width; c += tpr) {
                const float dy = lds_elem<T>(g, c), u = lds_elem<T>(h, c) * rs;
                const float wg = dy * load_weight<T, 1>(p.w, p.w_f32 != 0, c).p[0];
                dw[c] = fmaf(dy, u, dw[c]);
                dx[c] = from_f32<T>(fmaf(u, m, fmaf(wg, rs, has_d ? lds_elem<T>(d, c) : 0.0f)));
            }
        }
        last = slot;
        if (++slot == ring.slots) { slot = 0; phase ^= 1u; }
    }
    if (!ok) let_copies_land();
    if (p.partial == nullptr) return;
    __syncthreads();
    for (int c = tid; c < width; c += int(blockDim.x * blockDim.y)) {
        float s = dw_rows[c];
        for (int y = 1; y < int(blockDim.y); ++y) s += dw_rows[y * width + c];
        p.partial[int64_t(blockIdx.x) * p.width + c] = s;
    }
}

// Rows of which the ring's shared memory does not hold two slots, or of more than
// 16384 elements: dx with one block per row (two passes over it, element by element),
// dweight's column sums by another kernel before it. On 16-byte boundaries these are
// 16-bit rows past 16384; fp32 rows from 4736 to 8192 elements, where two blocks share
// an SM, and from 9560 on with grad_h, from 7104 to 8192 and from 14336 on without (512 x 20000 bf16 with grad_h: 90.6 us for both; 512 x 16384 in the ring form 26.5).
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_backward_long_kernel(const NormBackwardParams p) {
    __shared__ float red[32];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *g = static_cast<const T *>(p.g) + row * p.ldg, *h = static_cast<const T *>(p.h) + row * p.ldh;
    const T *dh = p.dh != nullptr ? static_cast<const T *>(p.dh) + row * p.lddh : nullptr;
    const float rs = p.rstd[row];
    auto wg = [&](int64_t at) { return to_f32<T>(g[at]) * load_weight<T, 1>(p.w, p.w_f32 != 0, at).p[0]; };
    float dot = 0.0f;
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) dot = fmaf(wg(at), to_f32<T>(h[at]), dot);
    const float c = -rs * (row_sum<false>(dot, red) * rs * p.inv_width);
    for (int64_t at = threadIdx.x; at < p.width; at += blockDim.x) {
        const float d = dh != nullptr ? to_f32<T>(dh[at]) : 0.0f;
        static_cast<T *>(p.dx)[row * p.lddx + at] = from_f32<T>(fmaf(to_f32<T>(h[at]) * rs, c, fmaf(wg(at), rs, d)));
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
// each add every blockDim.y-th row, then the first adds theirs in order. Bound by
// latency (304 x 4096: 5.0 MB, 3.4 us of a call). The partials come from L2: this
// kernel may be on an SM before they are written, and with `late` reads them before its
// own wait, so they are neither data that stays the same while it runs (no restricted
// pointer, which would promise that) nor safe to take from an L1 that an earlier
// launch has filled.
constexpr int kPartGroups = 32;
__global__ void __launch_bounds__(32 * kPartGroups) sum_partials_kernel(const float *partial, float *out, int64_t parts,
                                                                        int64_t width, uint32_t late) {
    __shared__ float s[kPartGroups][33];
    griddep_enter(late);
    const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.0f;
    if (col < width) {
#pragma unroll 4
        for (int64_t r = threadIdx.y; r < parts; r += kPartGroups) v += __ldcg(partial + r * width + col);
    }
    s[threadIdx.y][threadIdx.x] = v;
    griddep_leave(late);
    __syncthreads();
    if (threadIdx.y != 0 || col >= width) return;
    for (int g = 1; g < kPartGroups; ++g) v += s[g][threadIdx.x];
    out[col] = v;
}

// Rows of no values: scale 1, mean 0 and rstd 1 / sqrt(eps), as rows of zeros have them. Each may be absent.
__global__ void __launch_bounds__(256) empty_rows_kernel(float *scale, float *mean, float *rstd, int64_t rows, float eps) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (row >= rows) return;
    if (scale != nullptr) scale[row] = 1.0f;
    if (mean != nullptr) mean[row] = 0.0f;
    if (rstd != nullptr) rstd[row] = rsqrtf(eps);
}

}  // namespace g16
