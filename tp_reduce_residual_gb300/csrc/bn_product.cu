// bn_product.cu -- the experts' product of 4-bit microscaled operands.
//
// For the rows m of group e (offsets[e] <= m < offsets[e + 1]) and n in [0, N):
//   out[m, n] = bf16(alpha * sum_k a[m, k] * w[e, n, k])
// with a and w codes times block scales (bn_fp4.cu), summed in 32 bits by the
// tensor core.  Rows of no group (before the first, past the last) are written as zeros.
//
// Weights are the tensor core's M operand and rows its N operand, so that the few
// rows an expert has in a decode batch cost a narrow product (N = 16 upwards)
// and each weight is read once.  Persistent CTAs walk the output tiles; stages of
// 256 values of K are filled by TMA (codes, 128-byte swizzle) and bulk copies
// (scales), one thread copies scales to tensor memory and issues the products
// (tcgen05, block-scaled), the output warps take the accumulator out as BF16,
// hand it back, and store it.
//
// Two shapes.  One CTA: tiles of 128 features by 128 rows, two accumulators.  A
// pair of CTAs (cta_group::2): tiles of 256 features by 256 rows, of which each
// CTA loads half the weights and half the rows; twice the products for the same
// bytes, because what bounds large groups is the filling of shared memory by TMA
// (60 bytes a cycle and SM here, 59.7 in a loop of copies from L2 alone, whatever the
// number in flight).
//
// Measured.  Few rows: the stream of weights bounds it; 100 tokens with 8 of 256
// experts (192 of them reached, 1.28 GB) 187 us, 6.9 TB/s; one token with 10 experts
// (94 MB, not in L2) 20 us, 4.7 TB/s: its 640 tiles are a little over four rounds of
// the device, so the fifth leaves most of it idle.
// Large groups: 4096 tokens with 8 of 64 experts, N = 4096, K = 5120: 247 us in a
// burst (5.6 PFLOP/s, tensor pipe 64 % active), 282 under the power cap at
// 1.5 GHz.  In SM cycles: products alone 362 thousand, with scale copies 377, with
// loads 428; tiles of 384 rows and weights prefetched into L2 were not faster.
#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"
#include "bn_tensor.cuh"

namespace bn {

using namespace dev;

namespace {

constexpr int kHalf = 128;              // features, and at most rows, that one CTA loads for a tile
constexpr int kTileBytes = 128;         // codes of a stage: 256 values of K
constexpr int kBoxRows = 32;            // rows of the smaller TMA box of the row operand
constexpr int kTmemColumns = 512;       // accumulators, scales from column 256 on
constexpr int kScaleColumn = 256;

template <bool PAIR>
struct Shape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kTile = PAIR ? 256 : 128;  // features, and rows, of an output tile
    static constexpr int kAccs = PAIR ? 1 : 2;      // accumulators of kTile columns
    static constexpr int kStep = PAIR ? 32 : 16;    // rows of a product are rounded up to this
    static constexpr int kStages = PAIR ? 5 : 6;
    static constexpr int kRowAtoms = kTile / 128;   // scale tiles of the row operand
    static constexpr int kOffB = kHalf * kTileBytes;
    static constexpr int kOffSA = 2 * kHalf * kTileBytes;
    static constexpr int kOffSB = kOffSA + 2048;
    static constexpr int kStageBytes = kOffSB + kRowAtoms * 2048;
    static constexpr int kOutWarps = PAIR ? 8 : 4;
    static constexpr int kThreads = 64 + 32 * kOutWarps;  // copies, products, output
    static constexpr int kScaleStride = 16 + 16 * kRowAtoms;  // tensor memory columns of a stage's scales
};

struct Maps {
    CUtensorMap a, a_small, w;   // codes: boxes of 128 (a_small: 32) rows by 128 bytes
    CUtensorMap a_scales, w_scales;  // scale tiles: boxes of a stage's chunks of 512 bytes of so many row tiles
};

// Shared-memory operand descriptor of scales: 32 rows of 16 bytes, no swizzle, 8
// rows apart by 128 bytes.
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}

// The tensor core's instructions, for one CTA or issued once for a pair.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

#define BN_PRODUCT(group, vec)                                                                                \
    asm volatile(                                                                                             \
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                                                     \
        "tcgen05.mma.cta_group::" group ".kind::mxf4nvf4.block_scale.scale_vec::" vec                         \
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb),      \
        "r"((uint32_t)accumulate) : "memory")

template <bool MX, bool PAIR>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, bool accumulate)
{
    if constexpr (PAIR && MX) BN_PRODUCT("2", "2X");
    else if constexpr (PAIR) BN_PRODUCT("2", "4X");
    else if constexpr (MX) BN_PRODUCT("1", "2X");
    else BN_PRODUCT("1", "4X");
}
#undef BN_PRODUCT

template <bool MX, bool PAIR>
__global__ void __launch_bounds__(Shape<PAIR>::kThreads, 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ProductArgs p)
{
    using S = Shape<PAIR>;
    constexpr int kStages = S::kStages, kTile = S::kTile;
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
        const CUtensorMap *maps5[] = {&maps.w, &maps.w_scales, &maps.a, &maps.a_small, &maps.a_scales};
#pragma unroll
        for (int i = 0; i < 5; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(maps5[i]) : "memory");
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
    if (warp == 2) {
        tmem_alloc<PAIR>(smem_addr(&tmem_slot), kTmemColumns);
    }
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
    Tiles<kTile> tiles(start, cum, p.E, (unsigned)((p.N + kTile - 1) / kTile), (unsigned)unit, (unsigned)units);
    Tile t;
    const int nk = (p.K + 255) / 256;
    constexpr int kChunksPerStage = MX ? 2 : 4;

    // The copying and the issuing warp run their loops as a whole, so that loop
    // state stays in uniform registers; one elected thread does each stage's work.
    if (warp == 0) {
        const int wtiles = (p.N + 127) / 128;  // scale tiles of one expert
        uint32_t it = 0;  // stages filled
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const int f0 = t.f * kTile + (int)rank * kHalf;
            // this CTA's rows of the product's N operand: all, or half of the rounded count
            const int columns = (t.rows + S::kStep - 1) / S::kStep * S::kStep;
            const int nb = PAIR ? columns / 2 : columns, b0 = t.row0 + (PAIR ? (int)rank * nb : 0);
            const int boxes = nb > kHalf / 2 ? 0 : (nb + kBoxRows - 1) / kBoxRows;  // 0: one of kHalf rows
            const uint32_t codes = (uint32_t)(kHalf + (boxes ? boxes * kBoxRows : kHalf)) * kTileBytes;
            constexpr uint32_t kScaleBytes = kChunksPerStage * 512;
            const uint32_t bytes = S::kCtas * (codes + (1 + S::kRowAtoms) * kScaleBytes);
            // past the last features any scales will do
            const int sw = t.e * wtiles + min(f0 / kHalf, wtiles - 1);
            for (int k = 0; k < nk; ++k, ++it) {
                const uint32_t s = it % kStages;
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(empty + 8 * s, ((it / kStages) & 1u) ^ 1u, ctl));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t at = base + s * S::kStageBytes;
                    const uint32_t bar = PAIR ? mapa(full + 8 * s, 0) : full + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
                    const int x = k * kTileBytes, c = k * kChunksPerStage;
                    tma_2d<PAIR>(at, &maps.w, x, t.e * p.N + f0, bar);
                    if (boxes == 0)
                        tma_2d<PAIR>(at + S::kOffB, &maps.a, x, b0, bar);
                    for (int b = 0; b < boxes; ++b)
                        tma_2d<PAIR>(at + S::kOffB + b * kBoxRows * kTileBytes, &maps.a_small, x, b0 + b * kBoxRows, bar);
                    tma_3d<PAIR>(at + S::kOffSA, &maps.w_scales, 0, c, sw, bar);
                    // scale tiles past the group's rows are fetched too and not used
                    tma_3d<PAIR>(at + S::kOffSB, &maps.a_scales, 0, c, t.stile, bar);
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
                const uint32_t buf = n % S::kAccs;
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_empty + 8 * buf, ((n / S::kAccs) & 1u) ^ 1u, ctl));
                if (!ok) break;
                fence_after();
                const uint32_t columns = (uint32_t)((t.rows + S::kStep - 1) / S::kStep * S::kStep);
                // E2M1 operands, both with K along the row; E8M0 scales for MXFP4; N / 8, M / 16
                const uint32_t idesc = (1u << 7) | (1u << 10) | ((columns >> 3) << 17) | ((MX ? 1u : 0u) << 23) |
                                       ((kTile >> 4) << 24);
                const uint32_t d = tmem + buf * kTile;
                const bool two = S::kRowAtoms > 1 && columns > 128;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % kStages;
                    ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(full + 8 * s, (it / kStages) & 1u, ctl));
                    if (!ok) break;
                    fence_after();
                    const uint32_t at = base + s * S::kStageBytes;
                    const uint32_t sa = tmem + kScaleColumn + (it & 1u) * S::kScaleStride, sb = sa + 16u;
                    const uint64_t da = rows_desc(at), db = rows_desc(at + S::kOffB);
                    const uint64_t dsa = scales_desc(at + S::kOffSA), dsb = scales_desc(at + S::kOffSB);
                    auto scales = [&](int c) {
                        copy_scales<PAIR>(sa + 4 * c, dsa + 32 * c);
                        copy_scales<PAIR>(sb + 4 * S::kRowAtoms * c, dsb + 32 * c);
                        if (two) copy_scales<PAIR>(sb + 4 * S::kRowAtoms * c + 4, dsb + 32 * kChunksPerStage + 32 * c);
                    };
                    auto step = [&](int j) {
                        const uint32_t c = MX ? j >> 1 : j;
                        const uint32_t half = MX ? (j & 1u) * 2u : 0u;  // which 2 of the 4 scale bytes
                        product<MX, PAIR>(d, da + 2 * j, db + 2 * j, idesc | (half << 4) | (half << 29), sa + 4 * c,
                                          sb + 4 * S::kRowAtoms * c, k > 0 || j > 0);
                    };
                    // each step's scales just before its product
                    constexpr int kSteps = MX ? 2 : 1;  // steps of one scale chunk
                    if (elect_one()) {
                        if (k * 256 + 256 <= p.K) {  // unrolled: the issuing thread sets the pace
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (j % kSteps == 0) scales(j / kSteps);
                                step(j);
                            }
                        } else {
                            const int steps = (p.K - k * 256 + 63) / 64;
                            for (int j = 0; j < steps; ++j) {
                                if (j % kSteps == 0) scales(j / kSteps);
                                step(j);
                            }
                        }
                        commit<PAIR>(empty + 8 * s);
                        if (k == nk - 1) commit<PAIR>(acc_full + 8 * buf);
                    }
                }
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
        uint32_t n = 0;
        for (; tiles.next(t, lane); ++n) {
            const uint32_t buf = n % S::kAccs;
            // this warp's columns: at most 128
            const int cut = PAIR ? (t.rows + 31) / 32 * 16 : t.rows;
            const int lo = half ? cut : 0, hi = half ? t.rows : min(cut, t.rows);
            if (!__all_sync(kAll, wait_phase<PAIR, kPipe>(acc_full + 8 * buf, (n / S::kAccs) & 1u, ctl))) break;
            fence_after();
            // the whole tile as BF16 in registers, so that the next product can start
            uint32_t packed[8][8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (lo + 16 * b < hi) {
                    uint32_t v[16];
                    read16(tmem + ((uint32_t)(quad * 32) << 16) + buf * kTile + lo + 16 * b, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * i]) * p.alpha,
                                                                       __uint_as_float(v[2 * i + 1]) * p.alpha);
                        packed[b][i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) arrive_first(acc_empty + 8 * buf);
                else mbar_arrive(acc_empty + 8 * buf);
            }
            const int f = t.f * kTile + (int)rank * kHalf + quad * 32 + (lane & ~7);
            uint16_t *out = p.out + (long long)(t.row0 + (lane & 7)) * p.N + f;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (lo + 16 * b < hi) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = transpose8(packed[b] + 4 * h, lane);
                        const int c = lo + 16 * b + 8 * h;
                        if (c + (lane & 7) < hi && f < p.N)
                            *reinterpret_cast<uint4 *>(out + (long long)c * p.N) = v;
                    }
                }
            }
        }
        // rows of no group: before the first, and past the last
        const long long step = (long long)gridDim.x * (S::kThreads - 64);
        const auto zeros = [&](long long row, long long end) {
            const long long last = end * p.N / 8;
            for (long long i = row * p.N / 8 + (long long)blockIdx.x * (S::kThreads - 64) + (threadIdx.x - 64); i < last; i += step)
                reinterpret_cast<uint4 *>(p.out)[i] = make_uint4(0, 0, 0, 0);
        };
        zeros(0, start[0]);
        zeros(start[p.E], p.M);
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // the pair's products read both CTAs' shared memory
    if (warp == 2) {
        fence_after();
        tmem_free<PAIR>(tmem, kTmemColumns);
    }
}

cudaError_t make_maps(Maps *m, const ProductArgs &p, const uint8_t *a, const uint8_t *w, int fmt, int row_atoms)
{
    const auto codes = [&](CUtensorMap *map, const uint8_t *data, long long rows, int box) {
        return make_map<2>(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, data, {(cuuint64_t)p.K / 2, (cuuint64_t)rows},
                           {(cuuint32_t)kTileBytes, (cuuint32_t)box}, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const auto scales = [&](CUtensorMap *map, const uint8_t *data, long long tiles, int atoms) {
        return make_map<3>(map, CU_TENSOR_MAP_DATA_TYPE_INT64, 8, data, {64, (cuuint64_t)p.chunks, (cuuint64_t)tiles},
                           {64, fmt ? 2u : 4u, (cuuint32_t)atoms}, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    cudaError_t e = codes(&m->a, a, p.M, kHalf);
    if (e == cudaSuccess) e = codes(&m->a_small, a, p.M, kBoxRows);
    if (e == cudaSuccess) e = codes(&m->w, w, (long long)p.E * p.N, kHalf);
    if (e == cudaSuccess) e = scales(&m->a_scales, p.a_scales, p.a_tiles, row_atoms);
    if (e == cudaSuccess) e = scales(&m->w_scales, p.w_scales, (long long)p.E * ((p.N + 127) / 128), 1);
    return e;
}

template <bool PAIR>
cudaError_t launch_shape(const ProductArgs &p, const Maps &maps, int fmt, int sms, bool pdl, cudaStream_t st)
{
    using S = Shape<PAIR>;
    const auto smem = [](int E) { return 1024 + (size_t)S::kStages * S::kStageBytes + 2 * sizeof(int) * (size_t)(E + 1); };
    static KernelSetup setup[2];
    auto *k = fmt ? product_kernel<true, PAIR> : product_kernel<false, PAIR>;
    const cudaError_t e = setup[fmt](k, (int)smem(kMaxExperts));
    if (e != cudaSuccess) return e;
    const long long row_tiles = (long long)p.M / S::kTile + (p.E < p.M ? p.E : p.M);
    const long long most = row_tiles * ((p.N + S::kTile - 1) / S::kTile);
    const long long units = sms / S::kCtas;
    const int grid = (int)(most < units ? most : units) * S::kCtas;
    return launch_kernel(k, dim3((unsigned)grid), dim3(S::kThreads), smem(p.E), pdl, S::kCtas, st, maps, p);
}

// Which shape: rounds of tiles over the device, a pair's costing about 1.25 of a
// CTA's.  The groups' sizes are on the device; as many groups as rows allow are taken
// to be in use and to leave half a tile each.  Measured, one CTA / pairs (us), groups
// averaging r rows: 32 experts of 4096 x 4096, r = 48 52 / 52, 128 62 / 56, 256 95 /
// 72, 512 169 / 114; 32 of 1024 x 2048, r = 48 9.3 / 10.1, 160 13.6 / 14.7, 192 16.4 /
// 13.3; 8 of 512 x 1024, r = 512 6.5 / 8.4; one of 8192 x 8192, r = 256 15.1 / 15.8,
// 384 25.0 / 16.4.
bool take_pairs(const ProductArgs &p, int sms)
{
    const long long groups = p.E < p.M ? p.E : p.M;
    const auto rounds = [&](int tile, int units) {
        const long long even = p.M / tile + groups / 2, rows = even > groups ? even : groups;
        return (rows * ((p.N + tile - 1) / tile) + units - 1) / units;
    };
    return 5 * rounds(Shape<true>::kTile, sms / 2) < 4 * rounds(Shape<false>::kTile, sms);
}

}  // namespace

cudaError_t launch_product(const ProductArgs &p, const uint8_t *a, const uint8_t *w, int fmt, int sms, bool pdl,
                           cudaStream_t st)
{
    const cudaError_t ready = tensor_maps_ready();
    if (ready != cudaSuccess) return ready;
    const bool pair = take_pairs(p, sms);
    Maps maps;
    const cudaError_t e = make_maps(&maps, p, a, w, fmt, pair ? Shape<true>::kRowAtoms : Shape<false>::kRowAtoms);
    if (e != cudaSuccess) return e;
    return pair ? launch_shape<true>(p, maps, fmt, sms, pdl, st) : launch_shape<false>(p, maps, fmt, sms, pdl, st);
}

}  // namespace bn
