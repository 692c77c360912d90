// bn_linear.cu -- the experts' linear layers in 16 bits, and their gradients.
//
// For the rows m of group e (offsets[e] <= m < offsets[e + 1]), summed in 32 bits by
// the tensor core and rounded once:
//   forward          y[m, n] = sum_k x[rows[m], k] * w[e, n, k]
//   input gradient   dx[m, k] = sum_n dy[m, n] * w[e, n, k]
//   weight gradient  dw[e, n, k] = sum_m dy[m, n] * x[rows[m], k]
// y and dx of rows of no group are zeros, dw of an empty group too.
//
// One kernel in three modes.  Forward and input gradient: the output's contiguous
// dimension (n, k: features) is the tensor core's M operand and rows are its N operand, so
// that the few rows an expert has in a decode batch cost a narrow product and each weight is
// read once.  Weight gradient: n and k, so that a lane holds a part of a row of dw; its tiles
// are all whole and its sums short, so their way out counts.  What is
// summed over lies along the rows in memory (forward: both operands; input gradient: dy)
// or across them (w there, both operands of the weight gradient): the tensor core takes
// either, as a bit of its descriptor.
// Persistent CTAs walk the output tiles; stages of 64 values of the sum are filled by
// TMA (128-byte swizzle), one thread issues the products, the output warps take an
// accumulator out while the next one is filled.  A few rows given by index are fetched four
// at a time by their indexes; more go to their places in a workspace first.  A group's
// last rows in the weight gradient come by index too: one outside x reads zeros, where a
// box would bring in the next group's rows.
//
// Shapes, as in bn_product.cu: one CTA with tiles of 128 x 128, or a pair of CTAs
// (cta_group::2) with tiles of 256 x 256 of which each loads half of either operand.  Tall
// pairs take 512 rows, in both accumulators, with the same features: 48 bytes a cycle and SM
// to fill for 64, at no overlap of a tile's way out with the next.  Where tiles are too few
// for the device, clusters of CTAs each sum a part.
//
// Measured, a call alone (back to back under the power cap).  What one SM takes in (60 bytes a
// cycle) bounds pairs: 4096 tokens with 8 of 64 experts of 4096 x 5120 845 us (955; 1.63
// PFLOP/s), their tiles not full; one expert of 8192 x 8192 and as many rows 554 us (625) by
// tall pairs (1.99 PFLOP/s).  Rows by index cost their way to the workspace, 67 of 912 us (1001).
// Few rows: the stream of weights; 100 tokens with 8 of 256 experts of 6144 x 512 171 us
// (6.7 TB/s), one token with 10 of 512 x 8192 18.6 us (4.5).
// dw of 4096 tokens with 8 of 64, 5120 x 2048 (1.34 GB) 486 us (529); before its way out in
// whole lines 600 by transposed pieces of 16 bytes, 340 without any.  In FP32 (2.7 GB, sums of 512 rows
// in runs) 666 us (690) for 472 at the copy rate, and added to what is there 1110 (1095) for 874.
// Sums of more than 16384 values, in runs: 4096 rows of 131072 values by 4096 features 2.8 ms (2.5
// whole, by tall pairs), 4096 x 32768 x 8192 1.32 either way.
#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"
#include "bn_tensor.cuh"

namespace bn {

namespace {

constexpr int kHalf = 128;      // features, and at most rows, that one CTA loads for a tile
constexpr int kDepth = kSumStage;  // summed values of a stage: 128 bytes
constexpr int kLongLog = 8;     // 2^8 stages of y and dx are summed at a time by the tensor core: 16384 values
constexpr int kBoxRows = 16;    // rows of the smaller box
constexpr int kAtom = 64 * 128; // bytes of 64 features or rows by 64 values, where the sum runs across rows

enum Shape { kOne = 0, kPair = 1, kSplit = 2, kTall = 3 };

template <int SHAPE, bool WEIGHTS = false>
struct LinearShape {
    static constexpr bool kPairs = SHAPE == kPair || SHAPE == kTall;
    static constexpr int kCtas = kPairs ? 2 : 1;               // CTAs of one product
    static constexpr int kTile = kPairs ? 256 : 128;           // features of an output tile
    static constexpr int kBlock = SHAPE == kSplit ? 64 : kTile;  // rows of one product
    static constexpr int kBlocks = SHAPE == kTall ? 2 : 1;     // products of a tile
    static constexpr int kRows = kBlock * kBlocks;
    static constexpr int kStep = kPairs ? 32 : 16;             // rows of a product are rounded up to this
    static constexpr int kStages = SHAPE == kSplit ? 7 : SHAPE == kTall ? 4 : WEIGHTS ? 5 : 6;
    static constexpr int kOffQ = kHalf * 128;
    static constexpr int kBlockBytes = kBlock / kCtas * 128;
    static constexpr int kStageBytes = kOffQ + kBlocks * kBlockBytes;
    static constexpr int kColumns = 2 * kBlock;                // tensor memory: two accumulators
    static constexpr int kJoinBytes = SHAPE == kSplit ? (kRows + kMaxSplit) * kHalf * 4 : 0;  // parts of a split sum
    static constexpr int kOutWarps = kPairs ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kOutWarps;  // copies, products, output
    // 32 rows by 128 bytes of each output warp, on their way to a weight gradient
    static constexpr int kOutBytes = WEIGHTS ? kOutWarps * 4096 : 0;
    static constexpr size_t smem(int E) { return 1024 + (size_t)kStages * kStageBytes + kOutBytes + kJoinBytes + 2 * sizeof(int) * (size_t)(E + 1); }
};

struct LinearMaps {
    CUtensorMap p;                 // the features' operand: w, or dy
    CUtensorMap q, q_small;        // the rows' operand: x, or dy of the input gradient, in boxes of 128 (64) and 16 rows
    CUtensorMap p_rows, q_rows;    // row by row: dy and x of the weight gradient, x of the forward
    CUtensorMap p16, p4, q16, q4;  // the weight gradient's in boxes of 16 and 4 rows
    CUtensorMap out;               // an FP32 weight gradient that is added to, in boxes of 32 rows by 32
};

// The weight gradient's tiles: experts one after another, of one expert the tiles along a
// row (of K) of a feature tile (of N) next to each other.
template <int TILE>
class WeightTiles {
public:
    __device__ WeightTiles(int E, int K, int F, unsigned first, unsigned step)
        : tiles_r_((unsigned)(K + TILE - 1) / TILE), tiles_f_((unsigned)(F + TILE - 1) / TILE), K_(K), step_(step), id_(first),
          total_((unsigned long long)tiles_r_ * tiles_f_ * (unsigned)E)
    {
    }
    __device__ __forceinline__ bool next(Tile &t, int)
    {
        if (id_ >= total_) return false;
        const unsigned per = tiles_r_ * tiles_f_;
        const unsigned e = (unsigned)(id_ / per), local = (unsigned)(id_ - (unsigned long long)e * per);
        t.e = (int)e;
        t.f = (int)(local / tiles_r_);
        t.row0 = (int)(local - (unsigned)t.f * tiles_r_) * TILE;
        t.rows = min(TILE, K_ - t.row0);
        id_ += step_;
        return true;
    }

private:
    unsigned tiles_r_, tiles_f_;
    int K_;
    unsigned step_;
    unsigned long long id_, total_;
};

// Operand descriptor where the sum runs across the rows in memory: atoms of 64 values
// (128 bytes, swizzled) by 64 rows; the atoms 8 KB apart, 8 rows 1024 bytes.
__device__ __forceinline__ uint64_t across_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(kAtom >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <bool PAIR>
__device__ __forceinline__ void product16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                     "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                     "r"((uint32_t)accumulate) : "memory");
}

__device__ __forceinline__ uint32_t round16(float a, float b, bool fp16)
{
    if (fp16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// LONG: y or dx whose sums are cut into runs.
template <int MODE, int SHAPE, bool GATHER, bool LONG>
__global__ void __launch_bounds__(LinearShape<SHAPE>::kThreads, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearArgs p)
{
    using S = LinearShape<SHAPE, MODE == kWeightGrad>;
    constexpr bool PAIR = S::kPairs, SPLIT = SHAPE == kSplit;
    constexpr int kStages = S::kStages, kTile = S::kTile, kRows = S::kRows, kBlock = S::kBlock, kBlocks = S::kBlocks;
    constexpr bool kWeights = MODE == kWeightGrad, kRuns = kWeights || LONG;
    static_assert(!LONG || (!kWeights && kBlocks == 1), "runs take both accumulators in turn");
    constexpr bool kAcrossP = MODE != kForward, kAcrossQ = kWeights;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * kStages + 7];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int4 quads[32];  // row indexes of the copying warp
    float *parts = reinterpret_cast<float *>(raw + (base - smem_addr(raw)) + kStages * S::kStageBytes + S::kOutBytes);
    int *start = reinterpret_cast<int *>(parts) + S::kJoinBytes / 4;
    int *cum = start + p.E + 1;
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // full: the copies of a stage have landed (a pair's on the first CTA's barrier);
    // empty: the products have read it
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, done = acc_empty + 16;
    // a split sum: the parts of this CTA's rows have come; the other CTAs have read theirs
    const uint32_t joined = done + 8, joinable = joined + 8;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    // a unit: a CTA, a pair, or a cluster whose CTAs each sum a part
    const uint32_t parts_n = SPLIT ? (uint32_t)p.split : 1u, part = SPLIT ? cluster_ctarank() : 0u;
    const int ctas = SPLIT ? p.split : S::kCtas;
    const int unit = (int)blockIdx.x / ctas, units = (int)gridDim.x / ctas;

    griddep_launch_dependents();
    if (warp == 1 && elect_one()) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.p) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.q) : "memory");
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, S::kCtas * S::kOutWarps);
        }
        mbar_init(done, 1);
        if (SPLIT) {
            mbar_init(joined, 1);
            mbar_init(joinable, parts_n * S::kOutWarps);
        }
        fence_mbarrier_init();
    }
    if (warp == 2) tmem_alloc<PAIR>(smem_addr(&tmem_slot), S::kColumns);
    __syncwarp();
    if constexpr (PAIR || SPLIT) cluster_arrive();  // this CTA's barriers are ready
    griddep_wait();
    group_tiles<kRows>(p.offsets, p.M, p.E, S::kThreads, start, cum, p.err);
    fence_before();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_wait();  // and the other CTAs'
    fence_after();
    const uint32_t tmem = tmem_slot;

    Ctl ctl;
    ctl.abort = &abort_flag;
    ctl.err = p.err;
    ctl.spin = false;
    ctl.pipe_polls = kMaxSpins;
    auto tiles = [&]() {
        if constexpr (kWeights)
            return WeightTiles<kTile>(p.E, p.K, p.F, (unsigned)unit, (unsigned)units);
        else
            return Tiles<kRows, PAIR ? S::kStep : 0>(start, cum, p.E, (unsigned)((p.F + kTile - 1) / kTile), (unsigned)unit, (unsigned)units);
    }();
    Tile t = {};
    // the length of a tile's sum
    const auto depth = [&]() { return kWeights ? max(start[t.e + 1] - start[t.e], 0) : p.D; };
    // The tensor core drops what its FP32 sums cannot hold, always towards zero: 1e-9 of the
    // sum a value (2e-6 over 1024 rows of one sign, 1e-3 over 2^20).  A weight gradient in FP32
    // is summed so over 4 stages, one in 16 bits over 64, y and dx over 2^kLongLog, and those
    // sums are added with rounding.
    const int run_log = LONG ? kLongLog : p.out_fp32 ? 2 : 6, run_mask = (1 << run_log) - 1;
    // the stages of it that this CTA sums
    const auto stages = [&](int d, int &k0, int &k1) {
        const int nk = sum_stages(d);
        k0 = SPLIT ? (int)(part * (uint32_t)nk / parts_n) : 0;
        k1 = SPLIT ? (int)((part + 1) * (uint32_t)nk / parts_n) : nk;
    };
    // a tile's products, the rows of one, and its columns
    const auto blocks_of = [&]() { return kBlocks == 1 ? 1 : (t.rows + kBlock - 1) / kBlock; };
    const auto rows_of = [&](int b) { return kBlocks == 1 ? t.rows : min(kBlock, t.rows - b * kBlock); };
    const auto columns_of = [&](int b) { return (rows_of(b) + S::kStep - 1) / S::kStep * S::kStep; };

    // The copying and the issuing warp run their loops as a whole, so that loop
    // state stays in uniform registers; one elected thread does each stage's work,
    // or every lane fetches its four rows.
    if (warp == 0) {
        uint32_t it = 0;  // stages filled
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const int f0 = t.f * kTile + (int)rank * kHalf;
            // this CTA's rows of a product's N operand: all, or half of the rounded count
            const auto half_of = [&](int b) { return PAIR ? columns_of(b) / 2 : columns_of(b); };
            const int nb = half_of(0), b0 = t.row0 + (PAIR ? (int)rank * nb : 0);
            const int d = depth();
            int k0, k1;
            stages(d, k0, k1);
            const auto boxes_of = [&](int n) { return n > kHalf / 2 && !SPLIT ? 0 : (n + kBoxRows - 1) / kBoxRows; };  // 0: one of kHalf rows
            const int boxes = boxes_of(nb);
            // and of a second product
            const int nb2 = kBlocks > 1 && blocks_of() > 1 ? half_of(1) : 0, b2 = t.row0 + kBlock + (int)rank * nb2, boxes2 = boxes_of(nb2);
            const int q_atoms = nb > 64 ? 2 : 1;
            if constexpr (GATHER && !kWeights) {  // four rows a lane; places past the tile read zeros
                int v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 4 * lane + i;
                    v[i] = p.x_rows;
                    if (m < nb && b0 + m < t.row0 + t.rows) {
                        v[i] = __ldg(p.rows + b0 + m);
                        if ((unsigned)v[i] >= (unsigned)p.x_rows) {
                            atomicOr(p.err, BN_DEVERR_PERM_RANGE);
                            v[i] = 0;
                        }
                    }
                }
                __syncwarp();
                quads[lane] = make_int4(v[0], v[1], v[2], v[3]);
                __syncwarp();
            }
            for (int k = k0; k < k1; ++k, ++it) {
                const uint32_t s = it % kStages;
                if constexpr (GATHER && kWeights) {  // 16 places a quad: the same indexes for both atoms
                    int v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = k * kDepth + 4 * (lane & 15) + i;
                        v[i] = p.x_rows;
                        if (m < d) {
                            v[i] = __ldg(p.rows + start[t.e] + m);
                            if ((unsigned)v[i] >= (unsigned)p.x_rows) {
                                atomicOr(p.err, BN_DEVERR_PERM_RANGE);
                                v[i] = 0;
                            }
                        }
                    }
                    __syncwarp();
                    quads[lane] = make_int4(v[0], v[1], v[2], v[3]);
                    __syncwarp();
                }
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(empty + 8 * s, ((it / kStages) & 1u) ^ 1u, ctl));
                if (!ok) break;
                const uint32_t at = base + s * S::kStageBytes, q = at + S::kOffQ;
                const uint32_t bar = PAIR ? mapa(full + 8 * s, 0) : full + 8 * s;
                const int r0 = k * kDepth;
                if constexpr (!kWeights) {
                    if (elect_one()) {
                        uint32_t q_rows = GATHER ? (uint32_t)nb : (uint32_t)(boxes ? boxes * kBoxRows : kHalf);
                        if (kBlocks > 1 && nb2) q_rows += (uint32_t)(boxes2 ? boxes2 * kBoxRows : kHalf);
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, S::kCtas * ((uint32_t)kHalf + q_rows) * 128);
                        if constexpr (kAcrossP) {
                            tma_3d<PAIR>(at, &maps.p, f0, r0, t.e, bar);
                            tma_3d<PAIR>(at + kAtom, &maps.p, f0 + 64, r0, t.e, bar);
                        } else {
                            tma_3d<PAIR>(at, &maps.p, r0, f0, t.e, bar);
                        }
                        if constexpr (!GATHER) {
                            const auto block = [&](uint32_t to, int y, int n) {
                                if (n == 0) tma_2d<PAIR>(to, &maps.q, r0, y, bar);
                                for (int b = 0; b < n; ++b) tma_2d<PAIR>(to + b * kBoxRows * 128, &maps.q_small, r0, y + b * kBoxRows, bar);
                            };
                            block(q, b0, boxes);
                            if (kBlocks > 1 && nb2) block(q + S::kBlockBytes, b2, boxes2);
                        } else {
#pragma unroll 4
                            for (int i = 0; i < nb / 4; ++i) tma_rows<PAIR>(q + i * 512, &maps.q_rows, r0, quads[i], bar);
                        }
                    }
                } else {
                    const bool tail = r0 + kDepth > d;
                    // rows that the products read
                    const int m0 = start[t.e] + r0, live = tail ? (d - r0 + 15) / 16 * 16 : kDepth;
                    const uint32_t p_bytes = 2u * 128u * (uint32_t)live, q_bytes = (uint32_t)(q_atoms * 128 * live);
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, S::kCtas * (p_bytes + q_bytes));
                        // rows i and on of this stage, of dy and (unless rows come by index) of x
                        const auto box = [&](const CUtensorMap *mp, const CUtensorMap *mq, int i, int y) {
                            tma_2d<PAIR>(at + i * 128, mp, f0, y, bar);
                            tma_2d<PAIR>(at + kAtom + i * 128, mp, f0 + 64, y, bar);
                            if (!GATHER) {
                                tma_2d<PAIR>(q + i * 128, mq, b0, y, bar);
                                if (q_atoms == 2) tma_2d<PAIR>(q + kAtom + i * 128, mq, b0 + 64, y, bar);
                            }
                        };
                        if constexpr (GATHER) {
#pragma unroll 4
                            for (int i = 0; i < live / 4; ++i) {
                                const int4 y = quads[i];
                                tma_rows<PAIR>(q + i * 512, &maps.q_rows, b0, y, bar);
                                if (q_atoms == 2) tma_rows<PAIR>(q + kAtom + i * 512, &maps.q_rows, b0 + 64, y, bar);
                            }
                        }
                        if (!tail) {
                            box(&maps.p, &maps.q, 0, m0);
                        } else {
                            // 16 rows at a time while all are the group's, then 4 (past it: boxes
                            // outside the map, zeros); four that the group's end cuts, by index
                            const int left = d - r0;
                            int i = 0;
                            for (; i + 16 <= left; i += 16) box(&maps.p16, &maps.q16, i, m0 + i);
                            for (; i + 4 <= left; i += 4) box(&maps.p4, &maps.q4, i, m0 + i);
                            if (i < left) {
                                const int4 y = {m0 + i, i + 1 < left ? m0 + i + 1 : p.M, i + 2 < left ? m0 + i + 2 : p.M, p.M};
                                tma_rows<PAIR>(at + i * 128, &maps.p_rows, f0, y, bar);
                                tma_rows<PAIR>(at + kAtom + i * 128, &maps.p_rows, f0 + 64, y, bar);
                                if (!GATHER) {
                                    tma_rows<PAIR>(q + i * 128, &maps.q_rows, b0, y, bar);
                                    if (q_atoms == 2) tma_rows<PAIR>(q + kAtom + i * 128, &maps.q_rows, b0 + 64, y, bar);
                                }
                                i += 4;
                            }
                            for (; i < live; i += 4) box(&maps.p4, &maps.q4, i, p.M);
                        }
                    }
                }
            }
        }
        // no copy, and no arrival of a product, may be in flight into a CTA that leaves
        const uint32_t old = it > kStages ? it - kStages : 0;
        for (uint32_t i = old; ok && i < it; ++i)
            ok = wait_phase<PAIR, kPipe>(empty + 8 * (i % kStages), (i / kStages) & 1u, ctl);
        if (!ok) {  // after a timeout: wait for the copies, and where their barrier is the other CTA's, for a while
            for (uint32_t i = old; rank == 0 && i < it; ++i)
                wait_phase<false, kDrain>(full + 8 * (i % kStages), (i / kStages) & 1u, ctl);
            for (const long long t0 = clock64(); rank != 0 && clock64() - t0 < (1 << 22);) {}
        }
        __syncwarp();
    } else if (warp == 1) {
        // of a pair's CTAs the first issues the products
        if (rank == 0) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            while (ok && tiles.next(t, lane)) {
                // FP32 sums; the operands' type; which of them run across the rows; N / 8, M / 16
                const uint32_t type = p.dtype == BN_BF16 ? 1u : 0u;
                const uint32_t kind = (1u << 4) | (type << 7) | (type << 10) | ((kAcrossP ? 1u : 0u) << 15) |
                                      ((kAcrossQ ? 1u : 0u) << 16) | ((uint32_t)(kTile >> 4) << 24);
                const int blocks = blocks_of();
                // the accumulator of block b, in turn, once it has been taken out
                const auto accumulator = [&](int b) {
                    const uint32_t i = n + (uint32_t)b;
                    return __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_empty + 8 * (i & 1u), ((i >> 1) & 1u) ^ 1u, ctl));
                };
                ok = accumulator(0);
                if (!ok) break;
                fence_after();
                const int d = depth();
                int k0, k1;
                stages(d, k0, k1);
                for (int k = k0; k < k1; ++k, ++it) {
                    const uint32_t s = it % kStages;
                    const bool first = kRuns ? ((k - k0) & run_mask) == 0 : k == k0;
                    if (kRuns && first && k > k0) {  // on to the other accumulator
                        ++n;
                        ok = accumulator(0);
                        if (!ok) break;
                    }
                    ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(full + 8 * s, (it / kStages) & 1u, ctl));
                    if (!ok) break;
                    fence_after();
                    const uint32_t at = base + s * S::kStageBytes;
                    const uint64_t dp = kAcrossP ? across_desc(at) : rows_desc(at);
                    // 16 values: 32 bytes along a row, or 16 rows of 128 bytes
                    constexpr uint32_t kP = kAcrossP ? 128 : 2, kQ = kAcrossQ ? 128 : 2;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        if (b > 0 && b >= blocks) break;
                        if (b > 0 && k == k0) {
                            ok = accumulator(b);
                            if (!ok) break;
                            fence_after();
                        }
                        const uint32_t acc = tmem + ((n + b) & 1u) * kBlock;
                        const uint32_t idesc = kind | (((uint32_t)columns_of(b) >> 3) << 17);
                        const uint32_t from = at + S::kOffQ + b * S::kBlockBytes;
                        const uint64_t dq = kAcrossQ ? across_desc(from) : rows_desc(from);
                        if (elect_one()) {
                            if (k * kDepth + kDepth <= d) {  // unrolled: the issuing thread sets the pace
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    product16<PAIR>(acc, dp + kP * j, dq + kQ * j, idesc, !first || j > 0);
                            } else {
                                const int steps = (d - k * kDepth + 15) / 16;
                                for (int j = 0; j < steps; ++j)
                                    product16<PAIR>(acc, dp + kP * j, dq + kQ * j, idesc, !first || j > 0);
                            }
                            if (b == blocks - 1) commit<PAIR>(empty + 8 * s);
                            if (k == k1 - 1 || (kRuns && ((k - k0 + 1) & run_mask) == 0)) commit<PAIR>(acc_full + 8 * ((n + b) & 1u));
                        }
                    }
                    if (!ok) break;
                }
                if (kWeights && ok && k0 == k1 && elect_one()) commit<PAIR>(acc_full + 8 * (n & 1u));
                n += (uint32_t)blocks;
            }
            // Every product has ended before tensor memory is freed.  Only this CTA waits, so
            // only its barrier is told: an arrival at the other's could come after it left.
            if (elect_one()) {
                commit_here<PAIR>(done);
                wait_phase<false, kDrain>(done, 0, ctl);
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;         // the lanes of tensor memory that this warp reads
        const int half = (warp - 2) >> 2;  // of a pair's columns
        const bool fp16 = p.dtype == BN_FP16;
        uint32_t n = 0;
        // accumulator i is full; it has been taken out
        const auto taken = [&](uint32_t i) {
            const bool ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_full + 8 * (i & 1u), (i >> 1) & 1u, ctl));
            fence_after();
            return ok;
        };
        const auto release = [&](uint32_t i) {
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) arrive_first(acc_empty + 8 * (i & 1u));
                else mbar_arrive(acc_empty + 8 * (i & 1u));
            }
        };
        // a tile's accumulators: its products, or the runs of a sum
        int long_runs = 1;
        if (LONG) {
            int k0, k1;
            stages(p.D, k0, k1);
            long_runs = (k1 - k0 + run_mask) >> run_log;
        }
        const auto sums_of = [&]() { return kWeights ? sum_runs(depth(), run_log) : LONG ? long_runs : blocks_of(); };
        // the runs of a long sum from column lo to hi, added
        const auto add_runs = [&](int lo, int hi, auto &sums) {
            constexpr int kColumns = sizeof(sums) / sizeof(float);
#pragma unroll
            for (int i = 0; i < kColumns; ++i) sums[i] = 0.0f;
            for (int u = 0; u < long_runs; ++u) {
                if (u > 0 && !taken(n + u)) return false;
                const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + ((n + u) & 1u) * kBlock + lo;
#pragma unroll
                for (int b = 0; b < kColumns / 16; ++b) {
                    if (lo + 16 * b < hi) {
                        uint32_t v[16];
                        read16(from + 16 * b, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sums[16 * b + i] += __uint_as_float(v[i]);
                    }
                }
                release(n + u);
            }
            return true;
        };
        uint32_t tile = 0;  // tiles of long sums taken
        for (; tiles.next(t, lane); n += (uint32_t)sums_of()) {
            if (!taken(n)) break;
            const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), acc = lanes + (n & 1u) * kBlock;
            const long long row0 = t.row0;
            const int f0 = t.f * kTile + (int)rank * kHalf + quad * 32;
            if constexpr (SPLIT) {
                // Every CTA of the cluster finishes its share of the rows: the parts of a row
                // come to it from all of them and are added in the order of the sum.
                const int share = (columns_of(0) + (int)parts_n - 1) / (int)parts_n;
                const uint32_t turn = LONG ? tile++ : n;
                float sums[LONG ? kBlock : 16];
                if (LONG && !add_runs(0, t.rows, sums)) break;
                if (!__all_sync(kAll, wait_phase<true, kPipe>(joinable, (turn & 1u) ^ 1u, ctl))) break;
                const int r0 = (int)part * share, r1 = min(r0 + share, t.rows);
                if (quad == 0 && lane == 0) mbar_arrive_expect_tx(joined, parts_n * (uint32_t)max(r1 - r0, 0) * 512u);
                const uint32_t mine = smem_addr(parts) + 4u * (uint32_t)(quad * 32 + lane) + part * (uint32_t)share * 512u;
                int owner = 0, at = 0;  // the CTA that takes a row, and the row's place there
                uint32_t to = mapa(mine, 0), bar = mapa(joined, 0);
                const auto send16 = [&](int b, const uint32_t *v) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (16 * b + i < t.rows) send_cluster(to + (uint32_t)at * 512u, v[i], bar);
                        if (++at == share) {
                            at = 0;
                            owner = min(owner + 1, (int)parts_n - 1);
                            to = mapa(mine, (uint32_t)owner);
                            bar = mapa(joined, (uint32_t)owner);
                        }
                    }
                };
                if constexpr (LONG) {
#pragma unroll
                    for (int b = 0; b < kBlock / 16; ++b)
                        if (16 * b < t.rows) send16(b, reinterpret_cast<const uint32_t *>(sums) + 16 * b);
                } else {
#pragma unroll 1
                    for (int b = 0; 16 * b < t.rows; ++b) {
                        uint32_t v[16];
                        read16(acc + 16 * b, v);
                        send16(b, v);
                    }
                    release(n);
                }
                if (!__all_sync(kAll, wait_phase<true, kPipe>(joined, turn & 1u, ctl))) break;
                uint16_t *out = static_cast<uint16_t *>(p.out) + (row0 + r0) * p.F + f0 + lane;
                const float *from = parts + quad * 32 + lane;
                for (int r = r0; r < r1; ++r, out += p.F, from += 128) {
                    float sum = 0.0f;
                    for (int i = 0; i < (int)parts_n; ++i) sum += from[i * share * 128];
                    if (f0 + lane < p.F) *out = (uint16_t)round16(sum, 0.0f, fp16);
                }
                __syncwarp();
                if (lane < (int)parts_n) arrive_cluster(mapa(joinable, (uint32_t)lane));
            } else if constexpr (kWeights) {
                // A lane's row of dw, 128 bytes of it at a time, through shared memory (swizzled, so
                // that neither way has conflicts), and 4 whole lines a store from there; where it is
                // added to what dw holds, by TMA, which adds there (loads would wait for DRAM: 2.7
                // times as long).  Storing by TMA as well took 6 % longer: its rows queue with
                // those that come in.  Each half has 128 columns.
                const bool none = depth() == 0;  // an empty group: zeros, or nothing to add
                const int width = p.out_fp32 ? 32 : 64;
                const uint32_t box = base + kStages * S::kStageBytes + (uint32_t)(warp - 2) * 4096u;
                const int end = none && p.accumulate ? 0 : min(half * 128 + 128, t.rows);
                const int runs = sums_of();
                // 128 bytes of every lane's row, at column c
                const auto emit = [&](int c, const uint32_t *v) {
                    if (p.accumulate) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last box has been read
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 w = none ? make_uint4(0, 0, 0, 0) : make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        store_shared(box + (uint32_t)lane * 128u + (uint32_t)((i ^ (lane & 7)) << 4), w);
                    }
                    if (p.accumulate) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0 && f0 < p.F) {  // what lies past the matrix is not added
                            asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(&maps.out),
                                         "r"(t.row0 + c), "r"(f0), "r"(t.e), "r"(box) : "memory");
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                        return;
                    }
                    __syncwarp();
                    const int k = t.row0 + c + (lane & 7) * (width / 8);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3);
                        const uint4 w = load_shared(box + (uint32_t)r * 128u + (uint32_t)(((lane ^ r) & 7) << 4));
                        const long long at = ((long long)t.e * p.F + f0 + r) * p.K + k;
                        if (f0 + r < p.F && k < p.K)
                            *reinterpret_cast<uint4 *>(static_cast<char *>(p.out) + (p.out_fp32 ? 4 * at : 2 * at)) = w;
                    }
                };
                if (runs == 1) {
                    for (int c = half * 128; c < end; c += width) {
                        uint32_t v[32];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t x[16];
                            if (p.out_fp32) {
                                read16(acc + c + 16 * b, x);
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[16 * b + i] = x[i];
                            } else {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    read16(acc + c + 32 * b + 16 * h, x);
#pragma unroll
                                    for (int i = 0; i < 8; ++i)
                                        v[16 * b + 8 * h + i] = round16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), fp16);
                                }
                            }
                        }
                        if (c + width >= end) release(n);
                        emit(c, v);
                    }
                    if (half * 128 >= end) release(n);
                } else {
                    float sums[128];
                    bool ok = true;
#pragma unroll
                    for (int i = 0; i < 128; ++i) sums[i] = 0.0f;
                    for (int u = 0; u < runs; ++u) {
                        ok = u == 0 || taken(n + u);
                        if (!ok) break;
                        const uint32_t from = lanes + ((n + u) & 1u) * kBlock + half * 128;
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            if (half * 128 + 16 * b < end) {
                                uint32_t x[16];
                                read16(from + 16 * b, x);
#pragma unroll
                                for (int i = 0; i < 16; ++i) sums[16 * b + i] += __uint_as_float(x[i]);
                            }
                        }
                        release(n + u);
                    }
                    if (!ok) break;
                    if (p.out_fp32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (half * 128 + 32 * q < end) emit(half * 128 + 32 * q, reinterpret_cast<const uint32_t *>(sums) + 32 * q);
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = round16(sums[64 * q + 2 * i], sums[64 * q + 2 * i + 1], fp16);
                            if (half * 128 + 64 * q < end) emit(half * 128 + 64 * q, v);
                        }
                    }
                }
            } else {
                // the whole tile in 16 bits in registers, so that the next product can start
                const int f = f0 + (lane & ~7);
                // this warp's columns of a block: at most 128
                const auto range = [&](int q, int &lo, int &hi) {
                    const int rows = rows_of(q), cut = PAIR ? (rows + 31) / 32 * 16 : rows;
                    lo = half ? cut : 0;
                    hi = half ? rows : min(cut, rows);
                };
                uint32_t packed[kBlocks][8][8];
                bool ok = true;
                if constexpr (LONG) {
                    float sums[128];
                    int lo, hi;
                    range(0, lo, hi);
                    ok = add_runs(lo, hi, sums);
#pragma unroll
                    for (int b = 0; b < 8; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i) packed[0][b][i] = round16(sums[16 * b + 2 * i], sums[16 * b + 2 * i + 1], fp16);
                }
#pragma unroll
                for (int q = 0; q < (LONG ? 0 : kBlocks); ++q) {
                    if (q > 0 && q >= blocks_of()) break;
                    if (q > 0 && !taken(n + q)) {
                        ok = false;
                        break;
                    }
                    int lo, hi;
                    range(q, lo, hi);
                    const uint32_t from = lanes + ((n + q) & 1u) * kBlock + lo;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (lo + 16 * b < hi) {
                            uint32_t v[16];
                            read16(from + 16 * b, v);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                packed[q][b][i] = round16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), fp16);
                        }
                    }
                    release(n + q);
                }
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < kBlocks; ++q) {
                    if (q > 0 && q >= blocks_of()) break;
                    int lo, hi;
                    range(q, lo, hi);
                    uint16_t *out = static_cast<uint16_t *>(p.out) + (row0 + q * kBlock + (lane & 7)) * p.F + f;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (lo + 16 * b < hi) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 v = transpose8(packed[q][b] + 4 * h, lane);
                                const int c = lo + 16 * b + 8 * h;
                                if (c + (lane & 7) < hi && f < p.F) *reinterpret_cast<uint4 *>(out + (long long)c * p.F) = v;
                            }
                        }
                    }
                }
            }
        }
        if constexpr (!kWeights) {  // rows of no group: before the first, and past the last
            const long long step = (long long)gridDim.x * (S::kThreads - 64);
            uint4 *out = static_cast<uint4 *>(p.out);
            const auto zeros = [&](long long row, long long end) {
                const long long last = end * p.F / 8;
                for (long long i = row * p.F / 8 + (long long)blockIdx.x * (S::kThreads - 64) + (threadIdx.x - 64); i < last; i += step)
                    out[i] = make_uint4(0, 0, 0, 0);
            };
            zeros(0, start[0]);
            zeros(start[p.E], p.M);
        } else {
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the last boxes have been added
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR || SPLIT) cluster_sync_all();  // the others' products, or stores, reach this CTA's shared memory
    if (warp == 2) {
        fence_after();
        tmem_free<PAIR>(tmem, S::kColumns);
    }
}

cudaError_t make_linear_maps(LinearMaps *m, const LinearArgs &p, LinearMode mode, const void *x, long long ld, const void *w,
                             long long w_ld)
{
    constexpr CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT16;  // copied as they are
    const auto matrix = [&](CUtensorMap *map, const void *data, long long rows, long long width, long long stride, int box) {
        return make_map<2>(map, type, 2, data, {(cuuint64_t)width, (cuuint64_t)rows}, {64, (cuuint32_t)box},
                           CU_TENSOR_MAP_SWIZZLE_128B, (cuuint64_t)stride);
    };
    cudaError_t e;
    if (mode == kWeightGrad) {
        const long long n = p.rows ? p.x_rows : p.M;
        e = matrix(&m->p, w, p.M, p.F, w_ld, kDepth);
        if (e == cudaSuccess) e = matrix(&m->p_rows, w, p.M, p.F, w_ld, 1);
        if (e == cudaSuccess) e = matrix(&m->p16, w, p.M, p.F, w_ld, 16);
        if (e == cudaSuccess) e = matrix(&m->p4, w, p.M, p.F, w_ld, 4);
        if (e == cudaSuccess) e = matrix(&m->q, x, n, p.K, ld, kDepth);
        if (e == cudaSuccess) e = matrix(&m->q_rows, x, n, p.K, ld, 1);
        if (e == cudaSuccess) e = matrix(&m->q16, x, n, p.K, ld, 16);
        if (e == cudaSuccess) e = matrix(&m->q4, x, n, p.K, ld, 4);
        if (e == cudaSuccess && p.accumulate)
            e = make_map<3>(&m->out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.out, {(cuuint64_t)p.K, (cuuint64_t)p.F, (cuuint64_t)p.E}, {32, 32, 1},
                            CU_TENSOR_MAP_SWIZZLE_128B);
        m->q_small = m->q;
        return e;
    }
    const cuuint64_t inner = (cuuint64_t)(mode == kForward ? p.D : p.F), outer = (cuuint64_t)(mode == kForward ? p.F : p.D);
    e = make_map<3>(&m->p, type, 2, w, {inner, outer, (cuuint64_t)p.E}, {64, mode == kForward ? (cuuint32_t)kHalf : (cuuint32_t)kDepth, 1},
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (p.rows) {
        if (e == cudaSuccess) e = matrix(&m->q_rows, x, p.x_rows, p.D, ld, 1);
        m->q = m->q_small = m->p_rows = m->p16 = m->p4 = m->q16 = m->q4 = m->q_rows;
        return e;
    }
    if (e == cudaSuccess) e = matrix(&m->q, x, p.M, p.D, ld, kHalf);
    if (e == cudaSuccess) e = matrix(&m->q_small, x, p.M, p.D, ld, kBoxRows);
    m->p_rows = m->q_rows = m->p16 = m->p4 = m->q16 = m->q4 = m->q_small;
    return e;
}

// Output tiles, at most: the groups' sizes are on the device, and as many groups as rows
// allow may be in use.
template <int SHAPE>
long long most_tiles(const LinearArgs &p, int mode)
{
    using S = LinearShape<SHAPE>;
    const long long groups = p.E < p.M ? p.E : p.M;
    const long long rows = mode == kWeightGrad ? (long long)p.E * ((p.K + S::kRows - 1) / S::kRows)
                                               : ((long long)p.M + groups * (S::kRows - 1)) / S::kRows;
    return rows * ((p.F + S::kTile - 1) / S::kTile);
}

template <int MODE, int SHAPE, bool GATHER, bool LONG = false>
cudaError_t launch_shape(const LinearArgs &p, const LinearMaps &maps, int sms, bool pdl, cudaStream_t st)
{
    using S = LinearShape<SHAPE, MODE == kWeightGrad>;
    static KernelSetup setup;
    auto *k = linear_kernel<MODE, SHAPE, GATHER, LONG>;
    const cudaError_t e = setup(k, (int)S::smem(kMaxExperts));
    if (e != cudaSuccess) return e;
    const int ctas = SHAPE == kSplit ? p.split : S::kCtas;
    const long long most = most_tiles<SHAPE>(p, MODE);
    const long long units = SHAPE == kSplit ? resident_clusters(k, ctas, S::kThreads, S::smem(kMaxExperts), sms) : sms / ctas;
    const int grid = (int)(most < units ? most : units) * ctas;
    return launch_kernel(k, dim3((unsigned)grid), dim3(S::kThreads), S::smem(p.E), pdl, ctas, st, maps, p);
}

// Which shape.  Sums are split where tiles are too few for the device and a sum is long
// enough to pay for joining its parts (about 1.5 us, 8 stages).  Measured, whole / split (us, bytes at
// the copy rate first): 10 experts with one row, 512 x 8192 12.6: 29.3 / 19.6 (by 3); one
// expert, 16 rows, 4096 x 8192 10.0: 28.4 / 16.8 (4); 8 rows, 2048 x 8192 5.0: 28.3 / 13.8
// (8); 512 x 512 5.5 / 6.4 (2): too short.
// Pairs and their rows go by rounds of tiles over the device (groups are taken to leave half
// a tile each).  A pair's tile fills shared memory as long as a CTA's does, but has more to
// lose at a group's end: 4/3 of it (of few rounds 3/2).  A tall tile takes as long as two.
// Measured, one CTA / pairs / tall pairs (us): 4096 tokens with 8 of 64 experts of 4096 x
// 5120 1094 / 866 / 958, dx 1096 / 852 / 918; 2000 with 8 of 32, 1024 x 4096 135 / 119 / 133;
// one expert, 8192 x 8192 and as many rows 870 / 596 / 549, 1024 rows 135 / 96 / 88, 512
// 72 / 57 / 86; 1000 with 8 of 64, 4096 x 4096 387 / 363 / 406; 1024 with 2 of 8, 2048 x
// 2048 33 / 37 / 39.  A weight gradient's tiles are all whole: 333 with 4 of 16, 1024 x 2048
// 47 / 37; 4096 with 8 of 64, 5120 x 2048 913 / 612 (both before its way out in whole lines).
int choose_shape(LinearArgs &p, int mode, int sms)
{
    const long long groups = p.E < p.M ? p.E : p.M;
    const auto rounds = [&](int height, int tile, int units) {
        const long long even = p.M / height + groups / 2;
        const long long rows = mode == kWeightGrad ? (long long)p.E * ((p.K + height - 1) / height) : even > groups ? even : groups;
        return (rows * ((p.F + tile - 1) / tile) + units - 1) / units;
    };
    p.split = 1;
    if (mode == kWeightGrad) return rounds(256, 256, sms / 2) < rounds(128, 128, sms) ? kPair : kOne;
    const long long nk = sum_stages(p.D);
    p.split = choose_split(most_tiles<kSplit>(p, mode), nk, 8, (most_tiles<kOne>(p, mode) + sms - 1) / sms * nk, sms);
    if (p.split > 1) return kSplit;
    const long long one = rounds(128, 128, sms), pair = rounds(256, 256, sms / 2);
    if (one <= 8 ? 3 * pair >= 2 * one : 4 * pair >= 3 * one) return kOne;
    return 2 * rounds(512, 256, sms / 2) <= pair ? kTall : kPair;
}

// y and dx: a CTA's sum of more than 2^kLongLog stages is cut into runs.  (Runs leave no
// accumulator for a second product: tall pairs' long sums go to pairs.)
template <int MODE, bool LONG>
cudaError_t launch_sums(const LinearArgs &p, int shape, const LinearMaps &maps, int sms, bool pdl, cudaStream_t st)
{
    if constexpr (MODE == kForward) {
        if (p.rows && shape == kSplit) return launch_shape<MODE, kSplit, true, LONG>(p, maps, sms, pdl, st);
        if (p.rows) return launch_shape<MODE, kOne, true, LONG>(p, maps, sms, pdl, st);
    }
    if (shape == kSplit) return launch_shape<MODE, kSplit, false, LONG>(p, maps, sms, pdl, st);
    if (shape == kOne) return launch_shape<MODE, kOne, false, LONG>(p, maps, sms, pdl, st);
    if (shape == kPair || LONG) return launch_shape<MODE, kPair, false, LONG>(p, maps, sms, pdl, st);
    return launch_shape<MODE, LONG ? kPair : kTall, false, LONG>(p, maps, sms, pdl, st);
}

template <int MODE>
cudaError_t launch_mode(LinearArgs p, const LinearMaps &maps, int sms, bool pdl, cudaStream_t st)
{
    const int shape = choose_shape(p, MODE, sms);
    if constexpr (MODE == kWeightGrad) {
        if (p.rows) return launch_shape<MODE, kOne, true>(p, maps, sms, pdl, st);
        return shape == kPair ? launch_shape<MODE, kPair, false>(p, maps, sms, pdl, st) : launch_shape<MODE, kOne, false>(p, maps, sms, pdl, st);
    } else {
        return (sum_stages(p.D) + p.split - 1) / p.split > 1 << kLongLog ? launch_sums<MODE, true>(p, shape, maps, sms, pdl, st)
                                                                      : launch_sums<MODE, false>(p, shape, maps, sms, pdl, st);
    }
}

// Rows of x at their places, densely, and their scales if there are any.  A warp a row
// at a time, four 16-byte loads a lane in flight; the writes bound it (32768 rows of 10 KB
// from 4096 in 67 us alone, 5.0 TB/s written, 82 back to back).  With the groups' offsets an index
// outside x is an error between the first and the last alone; row 0 is placed for it anywhere.
__global__ void __launch_bounds__(256) place_rows_kernel(const uint4 *x, long long ld, int x_rows, const int32_t *rows, int M,
                                                         const int32_t *offsets, int E, int vectors, uint4 *out, const float *scales,
                                                         float *out_scales, unsigned *err)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warps = (int)gridDim.x * 8;
    for (long long m = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); m < M; m += warps) {
        int r = __ldg(rows + m);
        if ((unsigned)r >= (unsigned)x_rows) {
            const bool used = !offsets || (__ldg(offsets) <= m && m < __ldg(offsets + E));
            if (used && lane == 0) atomicOr(err, BN_DEVERR_PERM_RANGE);
            r = 0;
        }
        if (scales && lane == 0) out_scales[m] = __ldg(scales + r);
        const uint4 *from = x + (long long)r * ld;
        uint4 *to = out + m * vectors;
        int i = lane;
        for (; i + 96 < vectors; i += 128) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(from + i + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j) to[i + 32 * j] = v[j];
        }
        for (; i < vectors; i += 32) to[i] = __ldg(from + i);
    }
}

}  // namespace

cudaError_t launch_place_rows(const void *x, long long ld, int x_rows, const int32_t *rows, int M, const int32_t *offsets, int E, int K,
                              void *out, const float *scales, float *out_scales, unsigned *err, int sms, bool pdl, cudaStream_t st)
{
    const long long blocks = ((long long)M + 7) / 8, most = 8LL * sms;
    return launch_kernel(place_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, pdl, 1, st,
                         static_cast<const uint4 *>(x), ld / 8, x_rows, rows, M, offsets, E, K / 8, static_cast<uint4 *>(out), scales, out_scales,
                         err);
}

cudaError_t launch_linear(const LinearArgs &p, LinearMode mode, const void *x, long long ld, const void *w, long long w_ld, int sms,
                          bool pdl, cudaStream_t st)
{
    const cudaError_t ready = tensor_maps_ready();
    if (ready != cudaSuccess) return ready;
    LinearMaps maps = {};
    const cudaError_t e = make_linear_maps(&maps, p, mode, x, ld, w, w_ld);
    if (e != cudaSuccess) return e;
    switch (mode) {
    case kForward: return launch_mode<kForward>(p, maps, sms, pdl, st);
    case kInputGrad: return launch_mode<kInputGrad>(p, maps, sms, pdl, st);
    default: return launch_mode<kWeightGrad>(p, maps, sms, pdl, st);
    }
}

}  // namespace bn
