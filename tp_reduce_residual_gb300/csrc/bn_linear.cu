// bn_linear.cu -- the experts' linear layers in 16 bits, and their gradients.
//
// For the rows m of group e (offsets[e] <= m < offsets[e + 1]), summed in 32 bits by
// the tensor core and rounded once:
//   forward          y[m, n] = sum_k x[rows[m], k] * w[e, n, k]
//   input gradient   dx[m, k] = sum_n dy[m, n] * w[e, n, k]
//   weight gradient  dw[e, n, k] = sum_m dy[m, n] * x[rows[m], k]
// y and dx of rows of no group are zeros, dw of an empty group too.
//
// One kernel in three modes.  The output's contiguous dimension (n, k, k: features) is
// the tensor core's M operand and the other its N operand, so that the few rows an
// expert has in a decode batch cost a narrow product and each weight is read once, and
// so that all modes store alike.  What is summed over lies along the rows in memory
// (forward: both operands; input gradient: dy) or across them (w there, both operands
// of the weight gradient): the tensor core takes either, as a bit of its descriptor.
// Persistent CTAs walk the output tiles; stages of 64 values of the sum are filled by
// TMA (128-byte swizzle), one thread issues the products, the output warps take an
// accumulator out while the next one is filled.  Rows given by index are fetched four
// at a time by their indexes, so x is never copied.  A group's last rows in the weight
// gradient come the same way: an index outside x reads zeros, where a box would
// bring in the next group's rows.
//
// Two shapes, as in bn_product.cu: one CTA with tiles of 128 x 128, and a pair of CTAs
// (cta_group::2) with tiles of 256 x 256 of which each loads half of either operand.
#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"
#include "bn_tensor.cuh"

namespace bn {

namespace {

constexpr int kHalf = 128;      // features, and at most rows, that one CTA loads for a tile
constexpr int kDepth = 64;      // summed values of a stage: 128 bytes
constexpr int kBoxRows = 32;    // rows of the smaller box
constexpr int kAtom = 64 * 128; // bytes of 64 features or rows by 64 values, where the sum runs across rows

template <bool PAIR>
struct LinearShape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kTile = PAIR ? 256 : 128;  // features, and rows, of an output tile
    static constexpr int kStep = PAIR ? 32 : 16;    // rows of a product are rounded up to this
    static constexpr int kStages = 6;
    static constexpr int kOffQ = kHalf * 128;
    static constexpr int kStageBytes = 2 * kOffQ;
    static constexpr int kColumns = 2 * kTile;      // tensor memory: two accumulators
    static constexpr int kOutWarps = PAIR ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kOutWarps;  // copies, products, output
};

struct LinearMaps {
    CUtensorMap p;                 // the features' operand: w, or x
    CUtensorMap q, q_small;        // the rows' operand: x or dy, in boxes of 128 (64) and 32 rows
    CUtensorMap p_rows, q_rows;    // row by row: x (and dy) of the weight gradient, x of the forward
};

// The weight gradient's tiles: experts one after another, of one expert the row tiles
// (of N) of a feature tile next to each other.
template <int TILE>
class WeightTiles {
public:
    __device__ WeightTiles(int E, int N, int F, unsigned first, unsigned step)
        : tiles_r_((unsigned)(N + TILE - 1) / TILE), tiles_f_((unsigned)(F + TILE - 1) / TILE), N_(N), step_(step), id_(first),
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
        t.rows = min(TILE, N_ - t.row0);
        id_ += step_;
        return true;
    }

private:
    unsigned tiles_r_, tiles_f_;
    int N_;
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

template <int MODE, bool PAIR, bool GATHER>
__global__ void __launch_bounds__(LinearShape<PAIR>::kThreads, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearArgs p)
{
    using S = LinearShape<PAIR>;
    constexpr int kStages = S::kStages, kTile = S::kTile;
    constexpr bool kWeights = MODE == kWeightGrad;
    constexpr bool kAcrossP = MODE != kForward, kAcrossQ = kWeights;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    int *start = reinterpret_cast<int *>(raw + (base - smem_addr(raw)) + kStages * S::kStageBytes);
    int *cum = start + p.E + 1;
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // full: the copies of a stage have landed (a pair's on the first CTA's barrier);
    // empty: the products have read it
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, done = acc_empty + 16;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int unit = (int)blockIdx.x / S::kCtas, units = (int)gridDim.x / S::kCtas;

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
        fence_mbarrier_init();
    }
    if (warp == 2) tmem_alloc<PAIR>(smem_addr(&tmem_slot), S::kColumns);
    griddep_wait();
    group_tiles<kTile>(p.offsets, p.M, p.E, S::kThreads, start, cum, p.err);
    fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the pair's barriers are ready
    fence_after();
    const uint32_t tmem = tmem_slot;

    Ctl ctl;
    ctl.abort = &abort_flag;
    ctl.err = p.err;
    ctl.spin = false;
    ctl.pipe_polls = kMaxSpins;
    auto tiles = [&]() {
        if constexpr (kWeights)
            return WeightTiles<kTile>(p.E, p.N, p.F, (unsigned)unit, (unsigned)units);
        else
            return Tiles<kTile>(start, cum, p.E, (unsigned)((p.F + kTile - 1) / kTile), (unsigned)unit, (unsigned)units);
    }();
    Tile t = {};
    // the length of a tile's sum
    const auto depth = [&]() { return kWeights ? max(start[t.e + 1] - start[t.e], 0) : p.D; };
    const auto columns_of = [&]() { return (t.rows + S::kStep - 1) / S::kStep * S::kStep; };

    // The copying and the issuing warp run their loops as a whole, so that loop
    // state stays in uniform registers; one elected thread does each stage's work,
    // or every lane fetches its four rows.
    if (warp == 0) {
        uint32_t it = 0;  // stages filled
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const int f0 = t.f * kTile + (int)rank * kHalf;
            // this CTA's rows of the product's N operand: all, or half of the rounded count
            const int columns = columns_of();
            const int nb = PAIR ? columns / 2 : columns, b0 = t.row0 + (PAIR ? (int)rank * nb : 0);
            const int d = depth(), nk = (d + kDepth - 1) / kDepth;
            const int boxes = nb > kHalf / 2 ? 0 : (nb + kBoxRows - 1) / kBoxRows;  // 0: one of kHalf rows
            const int q_atoms = nb > 64 ? 2 : 1;
            int4 index = {};
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
                index = make_int4(v[0], v[1], v[2], v[3]);
            }
            for (int k = 0; k < nk; ++k, ++it) {
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
                    index = make_int4(v[0], v[1], v[2], v[3]);
                }
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(empty + 8 * s, ((it / kStages) & 1u) ^ 1u, ctl));
                if (!ok) break;
                const uint32_t at = base + s * S::kStageBytes, q = at + S::kOffQ;
                const uint32_t bar = PAIR ? mapa(full + 8 * s, 0) : full + 8 * s;
                const int r0 = k * kDepth;
                if constexpr (!kWeights) {
                    if (elect_one()) {
                        const uint32_t q_rows = GATHER ? (uint32_t)nb : (uint32_t)(boxes ? boxes * kBoxRows : kHalf);
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, S::kCtas * ((uint32_t)kHalf + q_rows) * 128);
                        if constexpr (kAcrossP) {
                            tma_3d<PAIR>(at, &maps.p, f0, r0, t.e, bar);
                            tma_3d<PAIR>(at + kAtom, &maps.p, f0 + 64, r0, t.e, bar);
                        } else {
                            tma_3d<PAIR>(at, &maps.p, r0, f0, t.e, bar);
                        }
                        if constexpr (!GATHER) {
                            if (boxes == 0) tma_2d<PAIR>(q, &maps.q, r0, b0, bar);
                            for (int b = 0; b < boxes; ++b)
                                tma_2d<PAIR>(q + b * kBoxRows * 128, &maps.q_small, r0, b0 + b * kBoxRows, bar);
                        }
                    }
                    if constexpr (GATHER) {
                        __syncwarp();
                        if (4 * lane < nb) tma_rows<PAIR>(q + lane * 512, &maps.q_rows, r0, index, bar);
                    }
                } else {
                    const bool tail = r0 + kDepth > d;
                    // rows that the products read
                    const int m0 = start[t.e] + r0, live = tail ? (d - r0 + 15) / 16 * 16 : kDepth;
                    const uint32_t p_bytes = 2u * 128u * (uint32_t)live, q_bytes = (uint32_t)(q_atoms * 128 * live);
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, S::kCtas * (p_bytes + q_bytes));
                        if (!GATHER && !tail) {
                            tma_2d<PAIR>(at, &maps.p, f0, m0, bar);
                            tma_2d<PAIR>(at + kAtom, &maps.p, f0 + 64, m0, bar);
                        }
                        if (!tail) {
                            tma_2d<PAIR>(q, &maps.q, b0, m0, bar);
                            if (q_atoms == 2) tma_2d<PAIR>(q + kAtom, &maps.q, b0 + 64, m0, bar);
                        }
                    }
                    __syncwarp();
                    const int quad = lane & 15, atom = lane >> 4, m = 4 * quad;
                    if (m < live && (GATHER || tail)) {
                        int4 own;  // the places themselves
                        own.x = r0 + m < d ? m0 + m : p.M;
                        own.y = r0 + m + 1 < d ? m0 + m + 1 : p.M;
                        own.z = r0 + m + 2 < d ? m0 + m + 2 : p.M;
                        own.w = r0 + m + 3 < d ? m0 + m + 3 : p.M;
                        tma_rows<PAIR>(at + atom * kAtom + quad * 512, &maps.p_rows, f0 + 64 * atom, GATHER ? index : own, bar);
                        if (tail && atom < q_atoms)
                            tma_rows<PAIR>(q + atom * kAtom + quad * 512, &maps.q_rows, b0 + 64 * atom, own, bar);
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
            for (; ok && tiles.next(t, lane); ++n) {
                const uint32_t buf = n & 1u;
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_empty + 8 * buf, ((n >> 1) & 1u) ^ 1u, ctl));
                if (!ok) break;
                fence_after();
                // FP32 sums; the operands' type; which of them run across the rows; N / 8, M / 16
                const uint32_t type = p.dtype == BN_BF16 ? 1u : 0u;
                const uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((kAcrossP ? 1u : 0u) << 15) |
                                       ((kAcrossQ ? 1u : 0u) << 16) | (((uint32_t)columns_of() >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
                const uint32_t acc = tmem + buf * kTile;
                const int d = depth(), nk = (d + kDepth - 1) / kDepth;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % kStages;
                    ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(full + 8 * s, (it / kStages) & 1u, ctl));
                    if (!ok) break;
                    fence_after();
                    const uint32_t at = base + s * S::kStageBytes;
                    const uint64_t dp = kAcrossP ? across_desc(at) : rows_desc(at);
                    const uint64_t dq = kAcrossQ ? across_desc(at + S::kOffQ) : rows_desc(at + S::kOffQ);
                    // 16 values: 32 bytes along a row, or 16 rows of 128 bytes
                    constexpr uint32_t kP = kAcrossP ? 128 : 2, kQ = kAcrossQ ? 128 : 2;
                    if (elect_one()) {
                        if (k * kDepth + kDepth <= d) {  // unrolled: the issuing thread sets the pace
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                product16<PAIR>(acc, dp + kP * j, dq + kQ * j, idesc, k > 0 || j > 0);
                        } else {
                            const int steps = (d - k * kDepth + 15) / 16;
                            for (int j = 0; j < steps; ++j)
                                product16<PAIR>(acc, dp + kP * j, dq + kQ * j, idesc, k > 0 || j > 0);
                        }
                        commit<PAIR>(empty + 8 * s);
                        if (k == nk - 1) commit<PAIR>(acc_full + 8 * buf);
                    }
                }
                if (kWeights && ok && nk == 0 && elect_one()) commit<PAIR>(acc_full + 8 * buf);
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
        for (; tiles.next(t, lane); ++n) {
            const uint32_t buf = n & 1u;
            // this warp's columns: at most 128
            const int cut = PAIR ? (t.rows + 31) / 32 * 16 : t.rows;
            const int lo = half ? cut : 0, hi = half ? t.rows : min(cut, t.rows);
            const bool none = kWeights && depth() == 0;  // an empty group
            if (!__all_sync(kAll, wait_phase<PAIR, kPipe>(acc_full + 8 * buf, (n >> 1) & 1u, ctl))) break;
            fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + buf * kTile;
            const long long row0 = kWeights ? (long long)t.e * p.N + t.row0 : t.row0;
            const int f0 = t.f * kTile + (int)rank * kHalf + quad * 32;
            const auto release = [&]() {
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) arrive_first(acc_empty + 8 * buf);
                    else mbar_arrive(acc_empty + 8 * buf);
                }
            };
            if (kWeights && p.out_fp32) {  // a lane's feature, row by row: 128 bytes a warp
                float *out = static_cast<float *>(p.out) + row0 * p.F + f0 + lane;
                const bool mine = f0 + lane < p.F;
                for (int c0 = lo; c0 < hi; c0 += 16) {
                    uint32_t v[16];
                    read16(acc + c0, v);
                    if (c0 + 16 >= hi) release();
                    if (mine) {
                        float old[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            old[i] = p.accumulate && c0 + i < hi ? out[(long long)(c0 + i) * p.F] : 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float sum = none ? 0.0f : __uint_as_float(v[i]);
                            if (c0 + i < hi) out[(long long)(c0 + i) * p.F] = p.accumulate ? old[i] + sum : sum;
                        }
                    }
                }
                if (lo >= hi) release();
                continue;
            }
            // the whole tile in 16 bits in registers, so that the next product can start
            uint32_t packed[8][8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (lo + 16 * b < hi) {
                    uint32_t v[16];
                    read16(acc + lo + 16 * b, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        packed[b][i] = none ? 0u : round16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), fp16);
                }
            }
            release();
            const int f = f0 + (lane & ~7);
            uint16_t *out = static_cast<uint16_t *>(p.out) + (row0 + (lane & 7)) * p.F + f;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (lo + 16 * b < hi) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = transpose8(packed[b] + 4 * h, lane);
                        const int c = lo + 16 * b + 8 * h;
                        if (c + (lane & 7) < hi && f < p.F) *reinterpret_cast<uint4 *>(out + (long long)c * p.F) = v;
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
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the pair's products read both CTAs' shared memory
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
        e = matrix(&m->p, x, n, p.F, ld, kDepth);
        if (e == cudaSuccess) e = matrix(&m->p_rows, x, n, p.F, ld, 1);
        if (e == cudaSuccess) e = matrix(&m->q, w, p.M, p.N, w_ld, kDepth);
        if (e == cudaSuccess) e = matrix(&m->q_rows, w, p.M, p.N, w_ld, 1);
        m->q_small = m->q;
        return e;
    }
    const cuuint64_t inner = (cuuint64_t)(mode == kForward ? p.D : p.F), outer = (cuuint64_t)(mode == kForward ? p.F : p.D);
    e = make_map<3>(&m->p, type, 2, w, {inner, outer, (cuuint64_t)p.E}, {64, mode == kForward ? (cuuint32_t)kHalf : (cuuint32_t)kDepth, 1},
                    CU_TENSOR_MAP_SWIZZLE_128B);
    if (p.rows) {
        if (e == cudaSuccess) e = matrix(&m->q_rows, x, p.x_rows, p.D, ld, 1);
        m->q = m->q_small = m->p_rows = m->q_rows;
        return e;
    }
    if (e == cudaSuccess) e = matrix(&m->q, x, p.M, p.D, ld, kHalf);
    if (e == cudaSuccess) e = matrix(&m->q_small, x, p.M, p.D, ld, kBoxRows);
    m->p_rows = m->q_rows = m->q_small;
    return e;
}

template <int MODE, bool PAIR, bool GATHER>
cudaError_t launch_mode(const LinearArgs &p, const LinearMaps &maps, int sms, bool pdl, cudaStream_t st)
{
    using S = LinearShape<PAIR>;
    const auto smem = [](int E) { return 1024 + (size_t)S::kStages * S::kStageBytes + 2 * sizeof(int) * (size_t)(E + 1); };
    static KernelSetup setup;
    auto *k = linear_kernel<MODE, PAIR, GATHER>;
    const cudaError_t e = setup(k, (int)smem(kMaxExperts));
    if (e != cudaSuccess) return e;
    const long long row_tiles = MODE == kWeightGrad ? (long long)p.E * ((p.N + S::kTile - 1) / S::kTile)
                                                    : (long long)p.M / S::kTile + (p.E < p.M ? p.E : p.M);
    const long long most = row_tiles * ((p.F + S::kTile - 1) / S::kTile);
    const long long units = sms / S::kCtas;
    const int grid = (int)(most < units ? most : units) * S::kCtas;
    return launch_kernel(k, dim3((unsigned)grid), dim3(S::kThreads), smem(p.E), pdl, S::kCtas, st, maps, p);
}

// Which shape: rounds of tiles over the device, a pair's tile costing about twice a
// CTA's for four times the products.
bool take_pairs(const LinearArgs &p, LinearMode mode, int sms)
{
    const auto rounds = [&](int tile, int units) {
        const long long groups = p.E < p.M ? p.E : p.M, even = p.M / tile + groups / 2;
        const long long rows = mode == kWeightGrad ? (long long)p.E * ((p.N + tile - 1) / tile) : even > groups ? even : groups;
        return (rows * ((p.F + tile - 1) / tile) + units - 1) / units;
    };
    return 2 * rounds(256, sms / 2) < rounds(128, sms);
}

template <int MODE>
cudaError_t launch_shapes(const LinearArgs &p, const LinearMaps &maps, int sms, bool pdl, cudaStream_t st)
{
    const bool pair = take_pairs(p, (LinearMode)MODE, sms);
    if constexpr (MODE != kInputGrad) {
        if (p.rows) return pair ? launch_mode<MODE, true, true>(p, maps, sms, pdl, st) : launch_mode<MODE, false, true>(p, maps, sms, pdl, st);
    }
    return pair ? launch_mode<MODE, true, false>(p, maps, sms, pdl, st) : launch_mode<MODE, false, false>(p, maps, sms, pdl, st);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &p, LinearMode mode, const void *x, long long ld, const void *w, long long w_ld, int sms,
                          bool pdl, cudaStream_t st)
{
    const cudaError_t ready = tensor_maps_ready();
    if (ready != cudaSuccess) return ready;
    LinearMaps maps;
    const cudaError_t e = make_linear_maps(&maps, p, mode, x, ld, w, w_ld);
    if (e != cudaSuccess) return e;
    switch (mode) {
    case kForward: return launch_shapes<kForward>(p, maps, sms, pdl, st);
    case kInputGrad: return launch_shapes<kInputGrad>(p, maps, sms, pdl, st);
    default: return launch_shapes<kWeightGrad>(p, maps, sms, pdl, st);
    }
}

}  // namespace bn
