// Host side of the gemm_ops C ABI (declared in include/gemm_ops.h): argument
// validation, the choice of kernel and launch shape, tensor maps and launches.
// Compiled in one translation unit with gemm_f16.cu (library.cu), whose device
// set-up, tensor-map, launch and status helpers it uses.
#include "gemm_ops.h"
#include "ops_linear.cuh"
#include "ops_norm.cuh"

namespace {

bool is_c_type(int32_t t) { return t >= GEMM_TYPE_F32 && t <= GEMM_TYPE_BF16; }
int type_bytes(int32_t t) { return t == GEMM_TYPE_F32 ? 4 : t == GEMM_TYPE_E4M3 ? 1 : 2; }
bool present(const gemm_matrix_t *m) { return m != nullptr && m->data != nullptr; }
bool element_aligned(const void *p, int32_t type) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(type_bytes(type) - 1)) == 0; }
uint64_t round128(uint64_t x) { return (x + 127u) / 128u * 128u; }
bool sizes_ok(int64_t a, int64_t b, int64_t c) { return a >= 0 && b >= 0 && c >= 0 && a <= kMaxDim && b <= kMaxDim && c <= kMaxDim; }

// A row-major matrix a call reads or writes element by element: [rows, cols] of
// `type`, unit column stride, rows that do not overlap.
gemm_status_t check_rows(const gemm_matrix_t *m, int64_t rows, int64_t cols) {
    if (m->stride_row < 1 || m->stride_col < 1) return GEMM_ERR_INVALID_ARG;
    if (!element_aligned(m->data, m->type)) return GEMM_ERR_INVALID_ARG;
    if (m->stride_col != 1 && cols > 1) return GEMM_ERR_UNSUPPORTED;
    if (rows > 1 && m->stride_row < cols) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

int device_state(DeviceState **ds) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || device_init(dev, ds) != cudaSuccess) return -1;
    return dev;
}

// launch_overlapped with a 2-D grid and block, and a cluster along x where
// `cluster` > 1.
template <typename... KArgs, typename... Args>
cudaError_t launch_shape(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, int cluster, cudaStream_t stream,
                         Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

// ------------------------------------------------------------------ per-device set-up
// linear_split's shapes: T = 16 << t rows of C, S = 1 << s CTAs along K.
constexpr int kSplitTs = 5, kSplitSs = 4;

// Ring depth by T: up to 64 rows the ring is kept under half the SM's shared
// memory, so that two CTAs share an SM and one's set-up and sum overlap the
// other's stream.
constexpr int split_stages(int T) { return T == 16 || T == 128 ? 3 : 2; }

// Done once per device: this file's kernels' shared-memory limits, and how many
// CTAs of each linear_split shape are resident at once (clusters of 8 do not fill
// every GPC).
struct OpsState {
    std::mutex mu;
    std::atomic<bool> ready{false};
    int split_slots[kSplitTs][kSplitSs];
};
OpsState g_ops[kMaxDevices];

template <typename K>
cudaError_t allow_smem(K *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

const OpsState *ops_init(int dev, int num_sms) {
    OpsState &o = g_ops[dev];
    if (o.ready.load(std::memory_order_acquire)) return &o;
    std::lock_guard<std::mutex> lock(o.mu);
    if (o.ready.load(std::memory_order_relaxed)) return &o;
    cudaError_t e = allow_smem(linear_pair<false, 2>, lin::PAIR_SMEM);
    if (e == cudaSuccess) e = allow_smem(linear_pair<false, 4>, lin::PAIR_SMEM);
    if (e == cudaSuccess) e = allow_smem(linear_pair<true, 2>, lin::PAIR_SMEM);
    if (e == cudaSuccess) e = allow_smem(linear_pair<true, 4>, lin::PAIR_SMEM);
    if (e == cudaSuccess) e = allow_smem(linear_split<false>, 232448);
    if (e == cudaSuccess) e = allow_smem(linear_split<true>, 232448);
    for (int t = 0; e == cudaSuccess && t < kSplitTs; ++t) {
        const int T = 16 << t;
        o.split_slots[t][0] = (T <= 64 ? 2 : 1) * num_sms;
        for (int s = 1; e == cudaSuccess && s < kSplitSs; ++s) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << s;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(unsigned(2 * num_sms) >> s << s);
            cfg.blockDim = dim3(lin::SPLIT_THREADS);
            cfg.dynamicSmemBytes = size_t(lin::split_smem(split_stages(T), T));
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, linear_split<false>, &cfg);
            // the query counts one CTA per SM for these shapes, also where two fit and run
            // (16384 x 4096 weights, 64 tokens, 128 clusters of 2: 25.6 us, in one round)
            o.split_slots[t][s] = (T <= 64 ? 2 : 1) * std::max(n, 1) << s;
        }
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return nullptr;
    }
    if (log_enabled())
        for (int t = 0; t < kSplitTs; ++t)
            std::fprintf(stderr, "[gemm_linear] T=%d resident CTAs by K slices 1/2/4/8: %d %d %d %d\n", 16 << t, o.split_slots[t][0],
                         o.split_slots[t][1], o.split_slots[t][2], o.split_slots[t][3]);
    o.ready.store(true, std::memory_order_release);
    return &o;
}

// ------------------------------------------------------------------ linear: operands
// An operand of the product as rows of contiguous elements: K-major (rows along
// M or N) or MN-major (rows along K).
struct Operand {
    const void *data;
    int64_t rows, inner, ld;
    int32_t type;
    bool mn_major;
    bool tma() const { return tma_ok(data, inner, ld, type_bytes(type)); }
    int64_t copy_ld() const { return int64_t(round128(uint64_t(inner) * type_bytes(type))) / type_bytes(type); }
    uint64_t copy_bytes() const { return uint64_t(rows) * uint64_t(copy_ld()) * type_bytes(type); }
};

// A [M,K] (`outer` = M, k along columns) or, with the strides exchanged, B^T [N,K].
gemm_status_t classify(const void *data, int32_t type, int64_t outer, int64_t K, int64_t stride_outer, int64_t stride_k,
                       Operand *op) {
    if (stride_outer < 1 || stride_k < 1) return GEMM_ERR_INVALID_ARG;
    if (!element_aligned(data, type)) return GEMM_ERR_INVALID_ARG;
    // a dimension of one element has no stride of its own
    if (stride_k == 1 || K == 1) {
        *op = Operand{data, outer, K, stride_outer, type, false};
    } else if (stride_outer == 1 || outer == 1) {
        if (type == GEMM_TYPE_E4M3) return GEMM_ERR_UNSUPPORTED;
        *op = Operand{data, K, outer, stride_k, type, true};
    } else {
        return GEMM_ERR_UNSUPPORTED;
    }
    if (K == 1 && stride_outer == 1 && type != GEMM_TYPE_E4M3) *op = Operand{data, 1, outer, stride_k, type, true};
    if (op->rows == 1) op->ld = op->copy_ld();
    return GEMM_OK;
}

// Copies up to two operands of one type onto 128-byte lines at dst_a / dst_b
// (nullptr: that one stays) and points them at the copies.
cudaError_t pack_operands(Operand *a, void *dst_a, Operand *b, void *dst_b, int num_sms, cudaStream_t stream) {
    const int32_t type = a->type;
    int64_t total = 0;
    auto blocks_for = [&](int64_t n) { return int(std::min<int64_t>(cdiv(n, 256), 8 * int64_t(num_sms))); };
    cudaError_t e = cudaSuccess;
    if (type == GEMM_TYPE_E4M3) {
        auto job = [](const Operand &o, void *dst) {
            PackBytesJob j;
            j.src = static_cast<const uint8_t *>(o.data);
            j.dst = static_cast<uint8_t *>(dst);
            j.rows = o.rows;
            j.inner = o.inner;
            j.ld_src = o.ld;
            j.ld_dst = o.copy_ld();
            j.gpr = (o.inner + 15) / 16;
            j.granules = dst != nullptr ? o.rows * j.gpr : 0;
            return j;
        };
        const PackBytesJob ja = job(*a, dst_a), jb = job(*b, dst_b);
        total = ja.granules + jb.granules;
        if (total > 0) e = launch_overlapped(pack_bytes_kernel, blocks_for(total), 256, 0, stream, ja, jb);
    } else {
        auto job = [](const Operand &o, void *dst) {
            PackJob j;
            j.src = static_cast<const uint16_t *>(o.data);
            j.dst = static_cast<uint16_t *>(dst);
            j.rows = o.rows;
            j.inner = o.inner;
            j.ld_src = o.ld;
            j.ld_dst = o.copy_ld();
            j.gpr = (o.inner + 7) / 8;
            j.granules = dst != nullptr ? o.rows * j.gpr : 0;
            return j;
        };
        const PackJob ja = job(*a, dst_a), jb = job(*b, dst_b);
        total = ja.granules + jb.granules;
        if (total > 0) e = launch_overlapped(pack_rows_kernel, blocks_for(total), 256, 0, stream, ja, jb);
    }
    for (Operand *o : {a, b}) {
        void *dst = o == a ? dst_a : dst_b;
        if (dst == nullptr) continue;
        o->ld = o->copy_ld();
        o->data = dst;
    }
    return e;
}

// The tensor map of an operand for stages of `kbs` k-blocks of 128 bytes and `mn`
// rows (or columns) per CTA, and how a stage is fetched through it (OperandLoad).
// Rows of the third dimension are whole pieces of one row of the operand: it is
// used only where the row's extent is a multiple of the piece, so that nothing
// but the operand is read.
bool encode_operand(CUtensorMap *map, OperandLoad *load, const Operand &o, int kbs, int mn) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    const int es = type_bytes(o.type), be = 128 / es;
    const CUtensorMapDataType dt = o.type == GEMM_TYPE_E4M3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : o.type == GEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int pieces = o.mn_major ? mn / be : kbs;
    load->mn = o.mn_major;
    load->mode = pieces == 1 ? kLoadOne : o.inner % be == 0 ? kLoadBoxed : kLoadLanes;
    load->copies = pieces;
    const uint32_t outer_box = uint32_t(o.mn_major ? kbs * be : mn);
    if (load->mode != kLoadBoxed)
        return encode_2d(map, dt, o.data, uint64_t(o.inner), uint64_t(o.rows), uint64_t(o.ld) * es, uint32_t(be), outer_box);
    const cuuint64_t dims[3] = {cuuint64_t(be), cuuint64_t(o.rows), cuuint64_t(o.inner / be)};
    const cuuint64_t strides[2] = {cuuint64_t(o.ld) * es, 128u};
    const cuuint32_t box[3] = {cuuint32_t(be), outer_box, cuuint32_t(pieces)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, dt, 3, const_cast<void *>(o.data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same descriptor fields as make_idesc with the operands' format: fp16 0,
// bf16 1 (kind::f16); e4m3 0 (kind::f8f6f4).
uint32_t linear_idesc(int32_t type, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
    const uint32_t f = type == GEMM_TYPE_BF16 ? 1u : 0u;
    return make_idesc(a_mn, b_mn, m, n) | (f << 7) | (f << 10);
}

// ------------------------------------------------------------------ linear: which kernel
struct LinearPlan {
    bool pair;
    int T, split, stages;   // linear_split
    int64_t whole, units;   // linear_pair: whole tiles, and units in all
    double split_us, pair_us;
    double split_load, pair_load;  // shares of the GPU's places that the launch takes
};

// Estimated microseconds, from what was measured on GB300. linear_split: set-up
// and end kSplitFixed, partial rows sent and summed at a time per row, the first
// loads back after kLatency, a stage of two k-blocks every kSplitStep, and the
// weights from DRAM at 6.2 bytes a picosecond, or at what the rings in flight carry
// where that is less (a ring's bytes every kRingTime), and from L2 at 11, once for
// every T rows.
// linear_pair: set-up and end kPairFixed, a k-block of one round every kPairStep
// (more where there is only one round, and hardly less for halves of tiles), and
// the weights at what the rings carry (4 x 16384 x 4096: pairs 35.4 us,
// linear_split 25.1; 200 x 16384 x 4096: 32.4 and 40.3).
constexpr double kLatency = 1.15, kDramBytes = 6.2e6, kL2Bytes = 11e6, kRingTime = 2.6, kSplitFixed = 3.0, kSplitCluster = 0.3,
                 kSplitSend = 0.008, kSplitRow = 0.018, kPairFixed = 3.9, kPairStep = 0.29, kPairFirst = 0.32, kPairHalf = 0.265,
                 kPairRingTime = 2.9, kKernelSwitch = 3.0, kSideBySide = 1.5, kHiddenStart = 2.0;
constexpr double kSplitStep[kSplitTs] = {0.36, 0.42, 0.45, 0.37, 0.80};

// linear_split's shape, rows per CTA T (an M-major A comes in chunks of 64 rows)
// and K slices S. (4096 x 4096 weights, one token: S = 8 8.4 us, 4 9.8, 2 11.6,
// 1 15.8; 256 tokens: T = 128, S = 2 14.6, T = 256, S = 4 16.6, pairs 21.1; 64 x
// 16384 x 4096: T = 64, S = 2 25.4, S = 4 29.9, T = 32, S = 1 28.9.)
double plan_split(int64_t M, int64_t N, int64_t num_kb, bool a_mn, const OpsState &o, LinearPlan *pl) {
    double best = 1e300;
    for (int t = a_mn ? 2 : 0; t < kSplitTs; ++t) {
        const int T = 16 << t;
        const int64_t tiles = cdiv(N, lin::SPLIT_ROWS) * cdiv(M, T);
        for (int s = 0; s < kSplitSs && (s == 0 || (int64_t(2) << s) <= num_kb); ++s) {
            const int64_t S = int64_t(1) << s, ctas = tiles * S;
            const double one = kSplitFixed + (s > 0 ? kSplitCluster : 0.0) + kSplitSend * T + kSplitRow * T / double(S);
            const double stream = kLatency + double(cdiv(cdiv(num_kb, lin::KPS), S) - 1) * kSplitStep[t];
            // a few CTAs more than fit start late but end soon after the others
            const double load = double(ctas) / o.split_slots[t][s];
            const double rounds = load <= 1.0 ? 1.0 : load <= 1.1 ? load : double(cdiv(ctas, o.split_slots[t][s]));
            const double rate = std::min(kDramBytes, double(ctas) * lin::split_ring(split_stages(T), T) / kRingTime);
            const double weights = double(N) * double(num_kb) * 128.0;
            const double moved = std::max(weights / rate, double(cdiv(M, T)) * weights / kL2Bytes);
            const double cost = rounds * one + std::max(rounds * stream, moved);
            if (cost < best) {
                best = cost;
                pl->T = T;
                pl->split = int(S);
                pl->split_load = load;
            }
        }
        if (T >= M) break;
    }
    pl->stages = split_stages(pl->T);
    return best;
}

// linear_pair's units: whole tiles for as many full rounds of the GPU's pairs as
// there are, then, where the tiles that remain fit into one round as halves, those
// (512 x 4096 x 4096: 64 halves 19.6 us, 32 tiles 23.0; 4000 x 5000 x 3000: 4 rounds
// of 76 and 32 halves 95.6 us, with 16 tiles 96.5).
double plan_pair(int64_t M, int64_t N, int64_t num_kb, int max_pairs, bool halves_allowed, LinearPlan *pl) {
    const int64_t tiles = cdiv(M, pair::TILE_M) * cdiv(N, pair::TILE_N), rest = tiles % max_pairs;
    const bool halves = halves_allowed && rest > 0 && 2 * rest <= max_pairs;
    pl->whole = halves ? tiles - rest : tiles;
    pl->units = pl->whole + (halves ? 2 * rest : 0);
    pl->pair_load = double(pl->units) / max_pairs;
    const double rounds = double(cdiv(pl->whole, max_pairs));
    const double step = rounds == 1.0 ? kPairFirst : rounds * kPairStep;
    // few rows: bound by how many bytes of weights the rings keep in flight
    const double rate = double(std::min<int64_t>(pl->units, max_pairs)) * 2 * lin::PAIR_STAGES * pair::B_STAGE_BYTES / kPairRingTime;
    return kPairFixed + std::max(double(num_kb) * (step + (halves ? kPairHalf : 0.0)), double(N) * double(num_kb) * 128.0 / rate);
}

LinearPlan plan_linear(int64_t M, int64_t N, int64_t num_kb, bool a_mn, bool alone, uint32_t flags, const DeviceState &ds,
                       const OpsState &o) {
    LinearPlan pl{};
    pl.split_us = plan_split(M, N, num_kb, a_mn, o, &pl);
    pl.pair_us = plan_pair(M, N, num_kb, ds.max_pairs, alone, &pl);
    pl.pair = (flags & GEMM_LINEAR_PAIR) || (!(flags & GEMM_LINEAR_SPLIT) && pl.pair_us <= pl.split_us);
    return pl;
}

bool c_map(CUtensorMap *map, const void *data, int32_t type, int64_t M, int64_t N, int64_t ld) {
    const int es = type_bytes(type);
    const CUtensorMapDataType dt = type == GEMM_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == GEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode_2d(map, dt, data, uint64_t(N), uint64_t(M), uint64_t(ld) * es, 128 / es, 32);
}

bool quad_aligned(const void *p, int64_t ld, int es) {
    return (reinterpret_cast<uintptr_t>(p) & uintptr_t(4 * es - 1)) == 0 && ld % 4 == 0;
}

// Two products of one call that do not need each other run one into the other:
// the second's tiles start where the first's last round leaves SMs idle
// (griddep_enter), so neither ends in halves of tiles. Not for many rounds of
// tiles, where little of that is left to gain and the power limit sets the pace
// (gradients, one into the other / one after the other: 257 x 1000 x 520 15.3 /
// 17.7 us, 2048 x 2048 x 1024 25.1 / 32.6, 4000 x 5000 x 3000, 5.7 rounds, 192 / 207,
// 4096 x 4096 x 4096, 6.7 rounds, 163 / 166, 8192 x 4096 x 4096, 10.1 rounds, 340 / 329).
constexpr double kOverlapRounds = 8.0;
enum class Order { kAlone, kFirst, kSecond };

// linear_pair's residual and C share one staging buffer per warp, which leaves the
// ring a sixth stage, where a tile's products take long enough to hide that (one
// buffer / two: 4096 x 8192 x 8192 e4m3 152 / 162 us, 8192 x 8192 x 4096 bf16 317 / 325,
// 2048 157 / 162, 1024 98.8 / 96.6; 8192 x 8192 x 2048 e4m3 111 / 108).
constexpr int kOneBufferKb = 32;

// The product and its epilogue on operands that TMA can describe. K >= 1.
gemm_status_t run_linear(const Operand &A, const Operand &B, int64_t M, int64_t N, int64_t K, const EpilogueParams &e,
                         uint32_t flags, const DeviceState *ds, const OpsState *ops, cudaStream_t stream,
                         Order order = Order::kAlone) {
    const bool f8 = A.type == GEMM_TYPE_E4M3;
    const int es = e.type == 0 ? 4 : 2;
    LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = M;
    p.N = N;
    p.e = e;
    p.num_kb = int32_t(cdiv(K, f8 ? 128 : 64));
    p.wait.timeout_ns = g_timeout_ns.load();
    p.wait.epoch = next_epoch();
    const LinearPlan pl = plan_linear(M, N, p.num_kb, A.mn_major, order == Order::kAlone, flags, *ds, *ops);
    p.late = order == Order::kSecond;
    CUtensorMap tmA, tmB, tmBhalf, tmC, tmR, tmP;
    cudaError_t err;
    if (pl.pair) {
        const int64_t nm = cdiv(M, pair::TILE_M), nn = cdiv(N, pair::TILE_N);
        if (nm * nn > kMaxDim / 2) return GEMM_ERR_UNSUPPORTED;
        std::memset(&tmC, 0, sizeof(tmC));
        tmR = tmP = tmC;
        if (!encode_operand(&tmA, &p.a, A, 1, pair::CTA_M) || !encode_operand(&tmB, &p.b, B, 1, pair::CTA_N) ||
            !encode_operand(&tmBhalf, &p.b_half, B, 1, pair::CTA_N / 2))
            return GEMM_ERR_CUDA;
        // a clipped TMA store writes whole 16-byte granules: C's and pre's rows must end on one
        const bool ends = (N * es) % 16 == 0;
        p.e.c_tma = ends && tma_ok(e.c, N, e.ldc, es);
        p.e.p_tma = e.pre != nullptr && ends && tma_ok(e.pre, N, e.ldp, es);
        p.e.r_tma = e.r != nullptr && tma_ok(e.r, N, e.ldr, es);
        if ((p.e.c_tma && !c_map(&tmC, e.c, int32_t(e.type), M, N, e.ldc)) ||
            (p.e.p_tma && !c_map(&tmP, e.pre, int32_t(e.type), M, N, e.ldp)) ||
            (p.e.r_tma && !c_map(&tmR, e.r, int32_t(e.type), M, N, e.ldr)))
            return GEMM_ERR_CUDA;
        p.sched.nm = int32_t(nm);
        p.sched.nn = int32_t(nn);
        p.sched.group_m = 8;
        p.sched.grouped = 1;
        p.num_units = int32_t(pl.units);
        p.whole = int32_t(pl.whole);
        p.idesc = linear_idesc(A.type, A.mn_major, B.mn_major, 2 * pair::CTA_M, pair::TILE_N);
        p.idesc_half = linear_idesc(A.type, A.mn_major, B.mn_major, 2 * pair::CTA_M, pair::TILE_N / 2);
        p.bufs = e.pre != nullptr || (e.r != nullptr && p.num_kb < kOneBufferKb) ? 2 : 1;
        p.stages = p.bufs == 2 ? 5 : 6;
        const dim3 grid(unsigned(2 * std::min<int64_t>(p.num_units, ds->max_pairs)));
        auto *kernel = f8 ? (es == 4 ? linear_pair<true, 4> : linear_pair<true, 2>)
                          : (es == 4 ? linear_pair<false, 4> : linear_pair<false, 2>);
        err = launch_shape(kernel, grid, dim3(lin::PAIR_THREADS), lin::PAIR_SMEM, 1, stream, tmA, tmB, tmBhalf, tmC, tmR,
                           tmP, p);
    } else {
        const int64_t nm = cdiv(M, pl.T), nn = cdiv(N, lin::SPLIT_ROWS);
        if (nm * nn > kMaxDim / lin::MAX_SPLIT) return GEMM_ERR_UNSUPPORTED;
        if (!encode_operand(&tmA, &p.a, A, lin::KPS, pl.T) || !encode_operand(&tmB, &p.b, B, lin::KPS, lin::SPLIT_ROWS))
            return GEMM_ERR_CUDA;
        p.sched.nm = int32_t(nm);
        p.sched.nn = int32_t(nn);
        p.num_units = int32_t(nm * nn);
        p.T = pl.T;
        p.tmem_cols = pl.T < 32 ? 32 : pl.T;
        p.split = pl.split;
        p.stages = pl.stages;
        // transposed product: the weights are the 128-row operand
        p.idesc = linear_idesc(A.type, B.mn_major, A.mn_major, lin::SPLIT_ROWS, uint32_t(pl.T));
        p.e.vec4 = quad_aligned(e.c, e.ldc, es) && (e.pre == nullptr || quad_aligned(e.pre, e.ldp, es)) &&
                   (e.r == nullptr || quad_aligned(e.r, e.ldr, es));
        const dim3 grid(unsigned(int64_t(p.num_units) * pl.split));
        err = launch_shape(f8 ? linear_split<true> : linear_split<false>, grid, dim3(lin::SPLIT_THREADS),
                           lin::split_smem(pl.stages, pl.T), pl.split, stream, tmB, tmA, p);
    }
    if (log_enabled())
        std::fprintf(stderr, "[gemm_linear] M=%lld N=%lld K=%lld kernel=%s T=%d split=%d stages=%d units=%d whole=%d\n", (long long)M,
                     (long long)N, (long long)K, pl.pair ? "pair" : "split", p.T, p.split, p.stages, p.num_units,
                     p.whole);
    return err == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// Workspace of two operands' copies: [A's][B's], each from a 256-byte boundary.
void copies_needed(const Operand &A, const Operand &B, uint64_t *a_bytes, uint64_t *b_bytes) {
    *a_bytes = A.tma() ? 0u : round256(A.copy_bytes());
    *b_bytes = B.tma() ? 0u : round256(B.copy_bytes());
}

gemm_status_t check_operands(const gemm_matrix_t *A, const gemm_matrix_t *B, int64_t M, int64_t N, int64_t K, Operand *a,
                             Operand *b) {
    if (A == nullptr || B == nullptr) return GEMM_ERR_INVALID_ARG;
    if (A->type != B->type || A->type < GEMM_TYPE_F16 || A->type > GEMM_TYPE_E4M3) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = classify(A->data, A->type, M, K, A->stride_row, A->stride_col, a);
    if (st == GEMM_OK) st = classify(B->data, B->type, N, K, B->stride_col, B->stride_row, b);
    return st;
}

gemm_status_t check_workspace(const void *ws, uint64_t bytes, uint64_t need, uintptr_t align) {
    if (need == 0) return GEMM_OK;
    if (ws == nullptr || bytes < need || (reinterpret_cast<uintptr_t>(ws) & (align - 1))) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_linear_workspace_size(const gemm_matrix_t *A, const gemm_matrix_t *B, int64_t M, int64_t N,
                                         int64_t K, uint64_t *bytes) {
    if (!sizes_ok(M, N, K)) return GEMM_ERR_INVALID_ARG;
    Operand a, b;
    const gemm_status_t st = check_operands(A, B, M, N, K, &a, &b);
    if (st != GEMM_OK) return st;
    uint64_t na = 0, nb = 0;
    if (M > 0 && N > 0 && K > 0) copies_needed(a, b, &na, &nb);
    if (bytes) *bytes = na + nb;
    return GEMM_OK;
}

gemm_status_t gemm_linear(const gemm_matrix_t *A, const gemm_matrix_t *B, const gemm_matrix_t *C,
                          const gemm_epilogue_t *ep, int64_t M, int64_t N, int64_t K, uint32_t flags, void *workspace,
                          uint64_t workspace_bytes, gemm_stream_t stream_) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(M, N, K) || C == nullptr) return GEMM_ERR_INVALID_ARG;
    if ((flags & ~GEMM_LINEAR_ALL_FLAGS) || flags == GEMM_LINEAR_ALL_FLAGS) return GEMM_ERR_INVALID_ARG;
    static const gemm_epilogue_t kPlain = {};
    if (ep == nullptr) ep = &kPlain;
    Operand a, b;
    gemm_status_t st = check_operands(A, B, M, N, K, &a, &b);
    if (st != GEMM_OK) return st;
    if (!is_c_type(C->type)) return GEMM_ERR_INVALID_ARG;
    if (ep->activation < GEMM_ACT_NONE || ep->activation > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
    if (ep->bias != nullptr && ((ep->bias_type != GEMM_TYPE_F32 && ep->bias_type != C->type) ||
                                !element_aligned(ep->bias, ep->bias_type)))
        return GEMM_ERR_INVALID_ARG;
    const bool f8 = A->type == GEMM_TYPE_E4M3;
    if ((ep->scale_a == nullptr) != (ep->scale_b == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (f8 != (ep->scale_a != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(ep->scale_a) | reinterpret_cast<uintptr_t>(ep->scale_b)) & 3u))
        return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    if (C->data == nullptr || (K > 0 && (A->data == nullptr || B->data == nullptr))) return GEMM_ERR_INVALID_ARG;
    for (const gemm_matrix_t *m : {C, &ep->residual, &ep->pre}) {
        if (m->data == nullptr) continue;
        if (m->type != C->type) return GEMM_ERR_INVALID_ARG;
        st = check_rows(m, M, N);
        if (st != GEMM_OK) return st;
    }
    uint64_t na = 0, nb = 0;
    if (K > 0) copies_needed(a, b, &na, &nb);
    st = check_workspace(workspace, workspace_bytes, na + nb, 128);
    if (st != GEMM_OK) return st;

    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    DeviceState *ds = nullptr;
    const int dev = device_state(&ds);
    const OpsState *ops = dev < 0 ? nullptr : ops_init(dev, ds->num_sms);
    if (ops == nullptr) return GEMM_ERR_CUDA;
    EpilogueParams e;
    std::memset(&e, 0, sizeof(e));
    e.c = C->data;
    e.ldc = C->stride_row;
    e.r = ep->residual.data;
    e.ldr = ep->residual.stride_row;
    e.pre = ep->pre.data;
    e.ldp = ep->pre.stride_row;
    e.bias = ep->bias;
    e.bias_type = uint32_t(ep->bias_type);
    e.sa = ep->scale_a;
    e.sb = ep->scale_b;
    e.type = uint32_t(C->type);
    e.act = uint32_t(ep->activation);
    if (K == 0) {
        LinearParams p;
        std::memset(&p, 0, sizeof(p));
        p.M = M;
        p.N = N;
        p.e = e;
        const int64_t strips = std::min<int64_t>(cdiv(N, 256), 1 << 20);
        const int64_t rows = std::min<int64_t>(M, std::max<int64_t>(1, 16 * int64_t(ds->num_sms) / strips));
        return launch_shape(linear_empty_kernel, dim3(unsigned(strips), unsigned(rows)), dim3(256), 0, 1, stream, p) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    if (na + nb > 0 && pack_operands(&a, na ? ws : nullptr, &b, nb ? ws + na : nullptr, ds->num_sms, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return run_linear(a, b, M, N, K, e, flags, ds, ops, stream);
}

}  // extern "C"

// ------------------------------------------------------------------ linear, backward
namespace {

// Column sums of D: each block sums a strip of 256 columns over rows_per_block
// rows, 64 where that gives the GPU enough blocks, fewer down to 8 (one per row
// group) where it does not.
struct GradPlan {
    int64_t rows_per_block, parts;
};
GradPlan plan_grad(int64_t M, int64_t N) {
    GradPlan g;
    g.rows_per_block = 64;
    while (g.rows_per_block > kGradGroups && cdiv(M, g.rows_per_block) * cdiv(N, 256) < 900) g.rows_per_block /= 2;
    if (cdiv(M, g.rows_per_block) > 512) g.rows_per_block = cdiv(cdiv(M, 512), kGradGroups) * kGradGroups;
    g.parts = cdiv(M, g.rows_per_block);
    return g;
}

struct BackwardSpace {
    uint64_t d, partial, a, b, total;
    int64_t ldd;
    bool store_d;
};

// The gradient's matrix D = G act'(pre) is stored where it differs from G or G
// cannot be read by TMA.
gemm_status_t backward_space(const gemm_matrix_t *G, const Operand &a, const Operand &b, int32_t act, bool need_dbias,
                             int64_t M, int64_t N, int64_t K, BackwardSpace *s) {
    std::memset(s, 0, sizeof(*s));
    if (M == 0 || N == 0) return GEMM_OK;
    s->store_d = act != GEMM_ACT_NONE || !tma_ok(G->data, N, G->stride_row, 2);
    s->ldd = (N + 63) / 64 * 64;
    if (s->store_d && K > 0) s->d = round256(uint64_t(M) * uint64_t(s->ldd) * 2u);
    if (need_dbias) {
        const GradPlan g = plan_grad(M, N);
        if (g.parts > 1) s->partial = round256(uint64_t(g.parts) * uint64_t(N) * 4u);
    }
    if (K > 0) copies_needed(a, b, &s->a, &s->b);
    s->total = s->d + s->partial + s->a + s->b;
    return GEMM_OK;
}

gemm_status_t check_backward(const gemm_matrix_t *G, const gemm_matrix_t *A, const gemm_matrix_t *B, int64_t M, int64_t N,
                             int64_t K, Operand *a, Operand *b) {
    if (!sizes_ok(M, N, K) || G == nullptr) return GEMM_ERR_INVALID_ARG;
    gemm_status_t st = check_operands(A, B, M, N, K, a, b);
    if (st != GEMM_OK) return st;
    if (A->type == GEMM_TYPE_E4M3) return GEMM_ERR_UNSUPPORTED;
    if (G->type != A->type) return GEMM_ERR_INVALID_ARG;
    return check_rows(G, M, N);
}

// A gradient is stored row by row or, like a weight kept as its transpose,
// column by column (*turned).
gemm_status_t check_gradient(const gemm_matrix_t *m, int64_t rows, int64_t cols, bool *turned) {
    if (!is_c_type(m->type)) return GEMM_ERR_INVALID_ARG;
    *turned = m->stride_col != 1 && m->stride_row == 1 && cols > 1;
    if (!*turned) return check_rows(m, rows, cols);
    const gemm_matrix_t t{m->data, m->stride_col, m->stride_row, m->type};
    return check_rows(&t, cols, rows);
}

cudaError_t zero_matrix(const gemm_matrix_t *m, bool turned, int64_t rows, int64_t cols, int num_sms, cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    if (turned) std::swap(rows, cols);
    const int blocks = int(std::min<int64_t>(cdiv(rows * cols, 256), 8 * int64_t(num_sms)));
    zero_c_kernel<<<blocks, 256, 0, stream>>>(m->data, rows, cols, turned ? m->stride_col : m->stride_row, type_bytes(m->type));
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grad(const GradParams &p, bool vec, int64_t parts, cudaStream_t stream) {
    const dim3 grid(unsigned(cdiv(p.N, 256)), unsigned(parts)), block(32, kGradGroups);
    return vec ? launch_shape(linear_grad_kernel<T, false>, grid, block, 0, 1, stream, p)
               : launch_shape(linear_grad_kernel<T, true>, grid, block, 0, 1, stream, p);
}

// Rows of a second 16-bit (or, `es` = 1, 8-bit) matrix that start at the same place in
// a granule of 8 elements as the first's, row by row.
bool same_places(const void *a, int64_t lda, const void *b, int64_t ldb, int es, int64_t rows) {
    return ((reinterpret_cast<uintptr_t>(a) / 2 - reinterpret_cast<uintptr_t>(b) / uintptr_t(es)) & 7u) == 0 &&
           (rows == 1 || (lda - ldb) % 8 == 0);
}

bool vec16(const void *p, int64_t ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

}  // namespace

extern "C" {

gemm_status_t gemm_linear_backward_workspace_size(const gemm_matrix_t *G, const gemm_matrix_t *A,
                                                  const gemm_matrix_t *B, int32_t activation, int32_t need_dbias,
                                                  int64_t M, int64_t N, int64_t K, uint64_t *bytes) {
    Operand a, b;
    gemm_status_t st = check_backward(G, A, B, M, N, K, &a, &b);
    if (st != GEMM_OK) return st;
    if (activation < GEMM_ACT_NONE || activation > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
    BackwardSpace s;
    st = backward_space(G, a, b, activation, need_dbias != 0, M, N, K, &s);
    if (st == GEMM_OK && bytes) *bytes = s.total;
    return st;
}

gemm_status_t gemm_linear_backward(const gemm_matrix_t *G, const gemm_matrix_t *A, const gemm_matrix_t *B,
                                   const gemm_matrix_t *pre, int32_t activation, const gemm_matrix_t *dA,
                                   const gemm_matrix_t *dB, float *dbias, int64_t M, int64_t N, int64_t K,
                                   uint32_t flags, void *workspace, uint64_t workspace_bytes, gemm_stream_t stream_) {
    // ---- validation (no GPU work before this point)
    Operand a, b;
    gemm_status_t st = check_backward(G, A, B, M, N, K, &a, &b);
    if (st != GEMM_OK) return st;
    if ((flags & ~GEMM_LINEAR_ALL_FLAGS) || flags == GEMM_LINEAR_ALL_FLAGS) return GEMM_ERR_INVALID_ARG;
    if (activation < GEMM_ACT_NONE || activation > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
    const bool has_pre = activation != GEMM_ACT_NONE;
    if (has_pre && M > 0 && N > 0) {
        if (!present(pre) || pre->type != G->type) return GEMM_ERR_INVALID_ARG;
        st = check_rows(pre, M, N);
        if (st != GEMM_OK) return st;
    }
    bool dA_t = false, dB_t = false;
    if (present(dA)) st = check_gradient(dA, M, K, &dA_t);
    if (st == GEMM_OK && present(dB)) st = check_gradient(dB, K, N, &dB_t);
    if (st != GEMM_OK) return st;
    if (reinterpret_cast<uintptr_t>(dbias) & 3u) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && G->data == nullptr) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && K > 0 && ((present(dA) && B->data == nullptr) || (present(dB) && A->data == nullptr)))
        return GEMM_ERR_INVALID_ARG;
    BackwardSpace s;
    st = backward_space(G, a, b, activation, dbias != nullptr, M, N, K, &s);
    if (st != GEMM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, s.total, 128);
    if (st != GEMM_OK) return st;

    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    DeviceState *ds = nullptr;
    const int dev = device_state(&ds);
    const OpsState *ops = dev < 0 ? nullptr : ops_init(dev, ds->num_sms);
    if (ops == nullptr) return GEMM_ERR_CUDA;
    if (M == 0 || N == 0) {  // empty sums
        if (present(dA) && zero_matrix(dA, dA_t, M, K, ds->num_sms, stream) != cudaSuccess) return GEMM_ERR_CUDA;
        if (present(dB) && zero_matrix(dB, dB_t, K, N, ds->num_sms, stream) != cudaSuccess) return GEMM_ERR_CUDA;
        if (dbias != nullptr && N > 0 && cudaMemsetAsync(dbias, 0, size_t(N) * 4u, stream) != cudaSuccess) return GEMM_ERR_CUDA;
        return GEMM_OK;
    }
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    void *ws_d = ws, *ws_a = ws + s.d + s.partial, *ws_b = ws + s.d + s.partial + s.a;
    float *ws_part = reinterpret_cast<float *>(ws + s.d);
    const bool products = K > 0 && (present(dA) || present(dB));

    // ---- operand copies; D and its column sums beside them
    const bool pack_a = products && present(dB) && s.a > 0, pack_b = products && present(dA) && s.b > 0;
    const bool packs = pack_a || pack_b;
    if (packs && pack_operands(&a, pack_a ? ws_a : nullptr, &b, pack_b ? ws_b : nullptr, ds->num_sms, stream) != cudaSuccess)
        return GEMM_ERR_CUDA;
    Operand d_rows{G->data, M, N, G->stride_row, G->type, false};
    const GradPlan gp = plan_grad(M, N);
    if ((s.store_d && products) || dbias != nullptr) {
        GradParams p;
        std::memset(&p, 0, sizeof(p));
        p.g = G->data;
        p.ldg = G->stride_row;
        p.pre = has_pre ? pre->data : nullptr;
        p.ldp = has_pre ? pre->stride_row : 0;
        p.d = s.store_d && products ? ws_d : nullptr;
        p.ldd = s.ldd;
        p.partial = dbias == nullptr ? nullptr : gp.parts > 1 ? ws_part : dbias;
        p.M = M;
        p.N = N;
        p.rows_per_block = gp.rows_per_block;
        p.act = uint32_t(activation);
        p.late = packs;
        const bool vec = N % 8 == 0 && vec16(p.g, p.ldg, 2) && (!has_pre || vec16(p.pre, p.ldp, 2));
        const cudaError_t e = G->type == GEMM_TYPE_F16 ? launch_grad<__half>(p, vec, gp.parts, stream)
                                                       : launch_grad<__nv_bfloat16>(p, vec, gp.parts, stream);
        if (e != cudaSuccess) return GEMM_ERR_CUDA;
        if (p.d != nullptr) {
            d_rows.data = ws_d;
            d_rows.ld = s.ldd;
        }
    }
    // the column sums' last step; after the products, it needs nothing of the one before it
    auto finish_dbias = [&] {
        if (dbias == nullptr || gp.parts == 1) return GEMM_OK;
        return launch_shape(sum_partials_kernel, dim3(unsigned(cdiv(N, 32))), dim3(32, kPartGroups), 0, 1, stream,
                            static_cast<const float *>(ws_part), dbias, gp.parts, N, uint32_t(products)) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    };
    if (!products) return finish_dbias();
    auto out = [](const gemm_matrix_t *m, bool turned) {
        EpilogueParams e;
        std::memset(&e, 0, sizeof(e));
        e.c = m->data;
        e.ldc = turned ? m->stride_col : m->stride_row;
        e.type = uint32_t(m->type);
        return e;
    };
    // An operand whose rows run along the summed dimension is MN-major. The forward
    // product summed over K; these sum over N (dA) and M (dB).
    auto turned = [](Operand o) {
        o.mn_major = !o.mn_major;
        return o;
    };
    const bool two = present(dA) && present(dB);
    bool overlap = false;
    if (two) {
        // One kernel for both, unless two pay for the change: a kernel whose code is not on
        // the SMs yet starts kKernelSwitch later (257 x 1000 x 512: 15.4 us with one of
        // each, 12.2 with one kernel; 2048 x 2048 x 1024: 30.4 and 26.4).
        const LinearPlan pa = plan_linear(dA_t ? K : M, dA_t ? M : K, cdiv(N, 64), dA_t ? turned(b).mn_major : d_rows.mn_major,
                                          false, 0, *ds, *ops);
        const LinearPlan pb = plan_linear(dB_t ? N : K, dB_t ? K : N, cdiv(M, 64), dB_t ? true : turned(a).mn_major, false, 0,
                                          *ds, *ops);
        overlap = pa.pair_load + pb.pair_load <= kOverlapRounds;
        // side by side where both fit the GPU at once, else the second's set-up is hidden
        auto both = [](double a, double b, double load) {
            return load <= 1.0 ? std::max(a, b) + kSideBySide : a + b - kHiddenStart;
        };
        const double pairs = both(pa.pair_us, pb.pair_us, pa.pair_load + pb.pair_load);
        const double splits = both(pa.split_us, pb.split_us, pa.split_load + pb.split_load);
        const double each = std::min(pa.pair_us, pa.split_us) + std::min(pb.pair_us, pb.split_us) + kKernelSwitch;
        if (flags == 0 && std::min(pairs, splits) <= each) flags = pairs <= splits ? GEMM_LINEAR_PAIR : GEMM_LINEAR_SPLIT;
    }
    if (present(dA)) {  // dA = D B^T, or its transpose B D^T
        const Operand w = turned(b);
        const Order order = overlap ? Order::kFirst : Order::kAlone;
        st = dA_t ? run_linear(w, d_rows, K, M, N, out(dA, true), flags, ds, ops, stream, order)
                  : run_linear(d_rows, w, M, K, N, out(dA, false), flags, ds, ops, stream, order);
        if (st != GEMM_OK) return st;
    }
    if (present(dB)) {  // dB = A^T D, or its transpose D^T A
        const Operand x = turned(a), d = turned(d_rows);
        const Order order = overlap ? Order::kSecond : Order::kAlone;
        st = dB_t ? run_linear(d, x, N, K, M, out(dB, true), flags, ds, ops, stream, order)
                  : run_linear(x, d, K, N, M, out(dB, false), flags, ds, ops, stream, order);
        if (st != GEMM_OK) return st;
    }
    return finish_dbias();
}

}  // extern "C"

// ------------------------------------------------------------------ RMS norm
namespace {

constexpr int64_t kNormParts = 608;  // blocks of the backward pass at most: 4 per SM

struct RowShape {
    int nv;        // loads of 8 elements per thread
    int tpr, rpb;  // threads per row, rows per block
    bool fits;     // the row fits its threads' registers
};

// One load per thread where 1024 threads hold the row so, else the fewest; with
// many rows `least` (four, two of fp32's twice as long ones), so that blocks are small and several on an SM are at different
// points of load, reduction and store. Short rows share a block of 256 threads.
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

// The persistent form's block: 256 threads (rows of up to 8192 elements), else
// 512; nv is the number of loads of 8 elements per thread. Two blocks of 256
// share an SM, each with half the shared memory for its ring.
struct RingPlan {
    bool ok;
    int tpr, rpb, nv;  // threads per row, rows per block side by side, loads per thread
    int rpt;           // rows a thread works on at a time
    int smem, grid;
    RingShape ring;
};

// `sums`: the backward pass, which adds up dweight over the block's rows: in
// shared memory behind the ring (any alignment), or, with vectors, in registers
// and at the end in the ring's place.
// `shift`: vectors of rows off 16-byte boundaries, which have up to 7 foreign
// elements in front.
RingPlan ring_plan(int64_t rows, int64_t width, int es, int arrays, bool vec, bool shift, bool sums, int num_sms) {
    RingPlan r{};
    const int threads = width + (shift ? 7 : 0) <= 8192 ? 256 : 512;
    const int64_t loads = cdiv(width + (shift ? 7 : 0), 8);
    r.nv = int(cdiv(loads, threads));
    if (r.nv > 4) return r;  // ok stays false
    r.tpr = int(cdiv(cdiv(loads, r.nv), 32) * 32);
    while (threads % r.tpr) r.tpr += 32;
    r.rpb = threads / r.tpr;
    r.ring.pitch = int((width * es + 15) / 16 * 16 + 16);
    // two rows at a time in the backward pass, where the registers and a slot's copies
    // (one lane each) allow it (8192 x 4096: 58.7 us with one, 54.4 with two)
    const int blocks_per_sm = threads == 256 ? 2 : 1, most = blocks_per_sm * num_sms;
    // shifted: a thread's rows are 8 k apart, or it has one row only
    const bool one_row = shift && cdiv(rows, r.rpb) <= most;
    r.rpt = sums && vec && r.nv <= 2 && arrays * r.rpb * 2 <= 32 && !one_row ? 2 : 1;
    r.ring.array_bytes = r.rpb * r.rpt * r.ring.pitch;
    r.ring.slot_bytes = arrays * r.ring.array_bytes;
    const int behind = sums && !vec ? int(r.rpb * width * 4) : 0;
    const int budget = (blocks_per_sm == 2 ? 113 : 226) * 1024 - 2048 - behind;
    r.ring.slots = std::min(kRingSlots, budget / r.ring.slot_bytes);
    if (r.ring.slots < 2 && r.rpt == 2) {
        r.rpt = 1;
        r.ring.array_bytes /= 2;
        r.ring.slot_bytes /= 2;
        r.ring.slots = std::min(kRingSlots, budget / r.ring.slot_bytes);
    }
    if (r.ring.slots < 2) return r;
    r.smem = r.ring.slots * r.ring.slot_bytes + behind;
    if (sums && vec && (r.rpb > 1 || shift)) r.smem = std::max(r.smem, r.rpb * r.tpr * 8 * std::max(r.nv, 2) * 4);
    r.grid = int(std::min<int64_t>(cdiv(rows, r.rpb * r.rpt), most));
    if (shift && !one_row) {
        if (most < 8) return r;
        r.grid = int(std::min<int64_t>(cdiv(r.grid, 8) * 8, most / 8 * 8));
    }
    r.ok = true;
    return r;
}

// Launches one ring kernel; its shared-memory limit is raised by its first
// launch on a device.
template <auto Kernel, typename P>
cudaError_t launch_ring(const RingPlan &r, const P &p, int dev, cudaStream_t stream) {
    static std::atomic<uint64_t> raised{0};  // one bit per device
    static_assert(kMaxDevices <= 64, "one bit per device");
    const uint64_t bit = uint64_t(1) << dev;
    if (!(raised.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = allow_smem(Kernel, 226 * 1024);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        raised.fetch_or(bit, std::memory_order_release);
    }
    return launch_shape(Kernel, dim3(unsigned(r.grid)), dim3(unsigned(r.tpr), unsigned(r.rpb)), r.smem, 1, stream, p, r.ring);
}

// Whether rms_norm_kernel's blocks take four loads per thread: rows of more than
// 2048 elements, several waves of them (one load or the fewest / four, bf16: 64 x
// 8192 2.1 / 2.8 us, 3000 x 2047 8.3 / 8.6, 3000 x 8192 25.6 / 19.5, 8000 x 8192 to 8 bits
// with a residual 78.7 / 68.1), more waves where the residual and its sum move as
// many bytes again (1000 x 5120 9.0 / 9.7, 3000 x 6144 27.0 / 24.7). The persistent
// ring of rows that the gradients use was slower here (8000 x 8192 to 8 bits 79.9).
bool many_rows(const NormParams &p, bool quant, int num_sms) {
    const int64_t waves = p.r != nullptr && !quant && p.width <= 8192 ? 16 : 4;
    return p.width > 2048 && p.rows >= waves * num_sms;
}

template <typename T, bool kQ>
cudaError_t launch_norm(const NormParams &p, bool vec, bool shift, int dev, int num_sms, cudaStream_t stream) {
    const int least = !many_rows(p, kQ, num_sms) ? 1 : sizeof(T) == 2 ? 4 : 2;
    if constexpr (sizeof(T) == 2) {
        const RowShape s = row_shape(p.width + 7, least);
        if (shift && s.fits) {
            auto *k = s.nv == 1   ? rms_norm_kernel<T, 8, 1, kQ, true>
                      : s.nv == 2 ? rms_norm_kernel<T, 8, 2, kQ, true>
                                  : rms_norm_kernel<T, 8, 4, kQ, true>;
            return launch_shape(k, dim3(unsigned(cdiv(p.rows, s.rpb))), dim3(unsigned(s.tpr), unsigned(s.rpb)), 0, 1, stream, p);
        }
    }
    if (!vec) {
        const RingPlan r = ring_plan(p.rows, p.width, int(sizeof(T)), p.r != nullptr ? 2 : 1, false, false, false, num_sms);
        if (r.ok) return launch_ring<rms_norm_rows_any_kernel<T, kQ>>(r, p, dev, stream);
    }
    const RowShape s = row_shape(p.width, least);
    if (!vec || !s.fits)
        return launch_shape(rms_norm_long_kernel<T>, dim3(unsigned(p.rows)), dim3(1024), 0, 1, stream, p, int32_t(kQ));
    auto *k = s.nv == 1   ? rms_norm_kernel<T, 8, 1, kQ, false>
              : s.nv == 2 ? rms_norm_kernel<T, 8, 2, kQ, false>
                          : rms_norm_kernel<T, 8, 4, kQ, false>;
    return launch_shape(k, dim3(unsigned(cdiv(p.rows, s.rpb))), dim3(unsigned(s.tpr), unsigned(s.rpb)), 0, 1, stream, p);
}

template <typename T, bool kShift>
cudaError_t launch_norm_backward_rows(const RingPlan &r, const NormBackwardParams &p, int dev, cudaStream_t stream) {
    if (r.nv == 1 && r.rpt == 2) return launch_ring<rms_norm_backward_rows_kernel<T, 1, 2, kShift>>(r, p, dev, stream);
    if (r.nv == 2 && r.rpt == 2) return launch_ring<rms_norm_backward_rows_kernel<T, 2, 2, kShift>>(r, p, dev, stream);
    if (r.nv <= 2) return launch_ring<rms_norm_backward_rows_kernel<T, 2, 1, kShift>>(r, p, dev, stream);
    if (r.nv == 3) return launch_ring<rms_norm_backward_rows_kernel<T, 3, 1, kShift>>(r, p, dev, stream);
    return launch_ring<rms_norm_backward_rows_kernel<T, 4, 1, kShift>>(r, p, dev, stream);
}

template <typename T>
cudaError_t launch_norm_backward(NormBackwardParams p, bool vec, bool shift, float *dweight, float *partial, int dev, int num_sms,
                                 cudaStream_t stream) {
    p.partial = dweight != nullptr ? partial : nullptr;
    int64_t parts;
    cudaError_t e;
    const int arrays = p.dh != nullptr ? 3 : 2;
    RingPlan r{};
    if constexpr (sizeof(T) == 2) {
        if (shift) r = ring_plan(p.rows, p.width, int(sizeof(T)), arrays, true, true, true, num_sms);
    }
    shift = r.ok;
    if (!r.ok) r = ring_plan(p.rows, p.width, int(sizeof(T)), arrays, vec, false, true, num_sms);
    if (r.ok) {
        parts = r.grid;
        if (vec) e = launch_norm_backward_rows<T, false>(r, p, dev, stream);
        else if (!shift) e = launch_ring<rms_norm_backward_rows_any_kernel<T>>(r, p, dev, stream);
        else if constexpr (sizeof(T) == 2) e = launch_norm_backward_rows<T, true>(r, p, dev, stream);
        else e = cudaErrorInvalidValue;  // shift is for 16-bit types
    } else {
        // dweight's sums first: they read grad, which dx may be written over
        const int64_t rows_per_block = cdiv(p.rows, kNormParts);
        parts = cdiv(p.rows, rows_per_block);
        e = cudaSuccess;
        if (dweight != nullptr)
            e = launch_shape(rms_norm_dweight_long_kernel<T>, dim3(unsigned(cdiv(p.width, 256)), unsigned(parts)), dim3(256),
                             0, 1, stream, p, rows_per_block);
        if (e == cudaSuccess)
            e = launch_shape(rms_norm_backward_long_kernel<T>, dim3(unsigned(p.rows)), dim3(1024), 0, 1, stream, p);
    }
    if (e == cudaSuccess && dweight != nullptr)
        e = launch_shape(sum_partials_kernel, dim3(unsigned(cdiv(p.width, 32))), dim3(32, kPartGroups), 0, 1, stream,
                         static_cast<const float *>(partial), dweight, parts, p.width, 0u);
    return e;
}

}  // namespace

extern "C" {

gemm_status_t gemm_rms_norm(const gemm_matrix_t *x, const gemm_matrix_t *residual, const void *weight,
                            int32_t weight_type, const gemm_matrix_t *y, const gemm_matrix_t *h, float *scale,
                            float *rstd, int64_t rows, int64_t width, float eps, gemm_stream_t stream_) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(rows, width, 0) || x == nullptr || y == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!is_c_type(x->type) || (y->type != x->type && y->type != GEMM_TYPE_E4M3)) return GEMM_ERR_INVALID_ARG;
    if (weight_type != GEMM_TYPE_F32 && weight_type != x->type) return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps <= 3.0e38f)) return GEMM_ERR_INVALID_ARG;
    const bool quant = y->type == GEMM_TYPE_E4M3;
    if (rows == 0 || width == 0) return GEMM_OK;
    if (x->data == nullptr || y->data == nullptr || weight == nullptr || quant != (scale != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (present(h) && !present(residual)) return GEMM_ERR_INVALID_ARG;
    if (!element_aligned(weight, weight_type) ||
        ((reinterpret_cast<uintptr_t>(scale) | reinterpret_cast<uintptr_t>(rstd)) & 3u))
        return GEMM_ERR_INVALID_ARG;
    for (const gemm_matrix_t *m : {x, residual, y, h}) {
        if (!present(m)) continue;
        if (m != y && m->type != x->type) return GEMM_ERR_INVALID_ARG;
        const gemm_status_t st = check_rows(m, rows, width);
        if (st != GEMM_OK) return st;
    }
    DeviceState *ds = nullptr;
    const int dev = device_state(&ds);
    if (dev < 0) return GEMM_ERR_CUDA;
    NormParams p;
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
    p.w_f32 = weight_type == GEMM_TYPE_F32;
    p.scale = scale;
    p.rstd = rstd;
    p.rows = rows;
    p.width = width;
    p.eps = eps;
    p.inv_width = 1.0f / float(width);
    p.wait.timeout_ns = g_timeout_ns.load();
    p.wait.epoch = next_epoch();
    const int es = type_bytes(x->type);
    bool vec = width % 8 == 0 && aligned16(weight) && vec16(p.x, p.ldx, es);
    if (p.r != nullptr) vec = vec && vec16(p.r, p.ldr, es);
    if (p.h != nullptr) vec = vec && vec16(p.h, p.ldh, es);
    vec = vec && (quant ? (reinterpret_cast<uintptr_t>(p.y) & 7u) == 0 && p.ldy % 8 == 0 : vec16(p.y, p.ldy, es));
    bool shift = !vec && es == 2 && weight_type == x->type && aligned16(weight) &&
                 same_places(p.x, p.ldx, p.y, p.ldy, quant ? 1 : 2, rows);
    if (p.r != nullptr) shift = shift && same_places(p.x, p.ldx, p.r, p.ldr, 2, rows);
    if (p.h != nullptr) shift = shift && same_places(p.x, p.ldx, p.h, p.ldh, 2, rows);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    auto launch = [&](auto *k) { return k(p, vec, shift, dev, ds->num_sms, stream); };
    const cudaError_t e =
        x->type == GEMM_TYPE_F32   ? launch(quant ? launch_norm<float, true> : launch_norm<float, false>)
        : x->type == GEMM_TYPE_F16 ? launch(quant ? launch_norm<__half, true> : launch_norm<__half, false>)
                                   : launch(quant ? launch_norm<__nv_bfloat16, true> : launch_norm<__nv_bfloat16, false>);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_rms_norm_backward_workspace_size(int64_t rows, int64_t width, uint64_t *bytes) {
    if (!sizes_ok(rows, width, 0)) return GEMM_ERR_INVALID_ARG;
    if (bytes) *bytes = uint64_t(std::min<int64_t>(rows, kNormParts)) * uint64_t(width) * 4u;
    return GEMM_OK;
}

gemm_status_t gemm_rms_norm_backward(const gemm_matrix_t *grad, const gemm_matrix_t *h, const void *weight,
                                     int32_t weight_type, const float *rstd, const gemm_matrix_t *grad_h,
                                     const gemm_matrix_t *dx, float *dweight, int64_t rows, int64_t width,
                                     void *workspace, uint64_t workspace_bytes, gemm_stream_t stream_) {
    // ---- validation (no GPU work before this point)
    if (!sizes_ok(rows, width, 0) || grad == nullptr || h == nullptr || dx == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!is_c_type(grad->type)) return GEMM_ERR_INVALID_ARG;
    if (weight_type != GEMM_TYPE_F32 && weight_type != grad->type) return GEMM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(dweight) & 3u) return GEMM_ERR_INVALID_ARG;
    if (width == 0) return GEMM_OK;
    if (rows > 0) {
        if (grad->data == nullptr || h->data == nullptr || dx->data == nullptr || weight == nullptr || rstd == nullptr)
            return GEMM_ERR_INVALID_ARG;
        if (!element_aligned(weight, weight_type) || (reinterpret_cast<uintptr_t>(rstd) & 3u)) return GEMM_ERR_INVALID_ARG;
        for (const gemm_matrix_t *m : {grad, h, grad_h, dx}) {
            if (!present(m)) continue;
            if (m->type != grad->type) return GEMM_ERR_INVALID_ARG;
            const gemm_status_t st = check_rows(m, rows, width);
            if (st != GEMM_OK) return st;
        }
    }
    uint64_t need = 0;
    if (dweight != nullptr) (void)gemm_rms_norm_backward_workspace_size(rows, width, &need);
    const gemm_status_t st = check_workspace(workspace, workspace_bytes, need, 16);
    if (st != GEMM_OK) return st;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    DeviceState *ds = nullptr;
    const int dev = device_state(&ds);
    if (dev < 0) return GEMM_ERR_CUDA;
    if (rows == 0) {
        if (dweight != nullptr && cudaMemsetAsync(dweight, 0, size_t(width) * 4u, stream) != cudaSuccess) return GEMM_ERR_CUDA;
        return GEMM_OK;
    }
    NormBackwardParams p;
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
    p.rstd = rstd;
    p.rows = rows;
    p.width = width;
    p.inv_width = 1.0f / float(width);
    p.wait.timeout_ns = g_timeout_ns.load();
    p.wait.epoch = next_epoch();
    const int es = type_bytes(grad->type);
    bool vec = width % 8 == 0 && aligned16(weight) && vec16(p.g, p.ldg, es) && vec16(p.h, p.ldh, es) &&
               vec16(p.dx, p.lddx, es);
    if (p.dh != nullptr) vec = vec && vec16(p.dh, p.lddh, es);
    bool shift = !vec && es == 2 && weight_type == grad->type && aligned16(weight) &&
                 same_places(p.g, p.ldg, p.h, p.ldh, 2, rows) && same_places(p.g, p.ldg, p.dx, p.lddx, 2, rows);
    if (p.dh != nullptr) shift = shift && same_places(p.g, p.ldg, p.dh, p.lddh, 2, rows);
    float *part = static_cast<float *>(workspace);
    const cudaError_t e = grad->type == GEMM_TYPE_F32   ? launch_norm_backward<float>(p, vec, shift, dweight, part, dev, ds->num_sms, stream)
                          : grad->type == GEMM_TYPE_F16 ? launch_norm_backward<__half>(p, vec, shift, dweight, part, dev, ds->num_sms, stream)
                                                        : launch_norm_backward<__nv_bfloat16>(p, vec, shift, dweight, part, dev, ds->num_sms, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // extern "C"
