// bn_product.cu -- the experts' product of 4-bit microscaled operands.
//
// For the rows m of group e (offsets[e] <= m < offsets[e + 1]) and n in [0, N):
//   out[m, n] = bf16(alpha * sum_k a[m, k] * w[e, n, k])
// with a and w codes times block scales (bn_fp4.cu), summed in 32 bits by the
// tensor core.  Rows past the last group are written as zeros.
//
// The tensor core computes a tile of 128 output features by up to 128 rows:
// weights are the M operand, rows the N operand, so that the few rows an expert
// has in a decode batch cost a narrow tile (N = 16 upwards) and each weight is
// read once.  Persistent CTAs, one per SM, walk the tiles; six stages of 256
// values of K are filled by TMA (codes, 128-byte swizzle) and bulk copies
// (scales), one thread copies scales to tensor memory and issues the products
// (tcgen05, block-scaled), four warps read the accumulators (two of 128 columns,
// so that a tile's output overlaps the next one's product), scale and store.
#include <mutex>

#include <cuda.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {

using namespace dev;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTile = 128;              // features, and rows, of an output tile
constexpr int kTileBytes = 128;         // codes of a stage: 256 values of K
constexpr int kBoxRows = 32;            // rows of one TMA box of the row operand
constexpr int kStagesP = 6;
constexpr int kOffB = kTile * kTileBytes;
constexpr int kOffSA = 2 * kTile * kTileBytes;
constexpr int kOffSB = kOffSA + 2048;
constexpr int kStageBytes = kOffSB + 2048;
constexpr int kThreads = 192;           // producer, product, 4 output warps
constexpr int kTmemColumns = 512;       // two accumulators, scales from column 256 on
constexpr int kScaleColumn = 256;

// One thread of a converged warp.  The product's and the copies' operands live in
// uniform registers; behind elect.sync the compiler knows that one thread runs.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

struct Sched {
    int tiles_f;      // feature tiles of an expert
    long long total;  // tiles of all experts
};

struct Tile {
    int e, f, row0, rows, stile;
};

// Tile `id`: experts in order; of one expert, the row tiles of a feature tile
// next to each other, so that CTAs that run together share its weights in L2.
__device__ __forceinline__ Tile tile_of(long long id, const Sched &s, const int *start, const int *cum, int E)
{
    const int tt = (int)(id / s.tiles_f);
    int lo = 0, hi = E;  // cum[lo] <= tt < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= tt) lo = mid; else hi = mid;
    }
    const int nt = cum[lo + 1] - cum[lo];
    const int local = (int)(id - (long long)cum[lo] * s.tiles_f);
    Tile t;
    t.e = lo;
    t.f = local / nt;
    const int r = local % nt;
    t.row0 = start[lo] + r * kTile;
    t.rows = min(kTile, start[lo + 1] - t.row0);
    t.stile = (start[lo] >> 7) + lo + r;
    return t;
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Shared-memory operand descriptors.  Codes: rows of 128 bytes, 128-byte
// swizzle, 8 rows apart by 1024 bytes.  Scales: 32 rows of 16 bytes, no
// swizzle, 8 rows apart by 128 bytes.
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <bool MX>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, bool accumulate)
{
    if constexpr (MX)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"((uint32_t)accumulate) : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void read16(uint32_t tmem, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(tmem) : "memory");
}

template <bool MX>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ ProductArgs p)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * kStagesP + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    int *start = reinterpret_cast<int *>(raw + (base - smem_addr(raw)) + kStagesP * kStageBytes);
    int *cum = start + p.E + 1;
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kStagesP, acc_full = empty + 8 * kStagesP,
                   acc_empty = acc_full + 16, done = acc_empty + 16;

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kStagesP; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 128);
        }
        mbar_init(done, 1);
        fence_mbarrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(kTmemColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    griddep_wait();
    // the groups' first rows and the row tiles before each group
    for (int e = threadIdx.x; e <= p.E; e += kThreads) {
        const int o = p.offsets ? __ldg(p.offsets + e) : e * p.M;
        if (o < 0 || o > p.M) atomicOr(p.err, BN_DEVERR_OFFSETS);
        start[e] = min(max(o, 0), p.M);
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        if (lane == 0) cum[0] = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.E) {
                n = start[e + 1] - start[e];
                if (n < 0) {  // a falling offset: an empty group
                    atomicOr(p.err, BN_DEVERR_OFFSETS);
                    n = 0;
                }
                n = (n + kTile - 1) / kTile;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kAll, n, o);
                if (lane >= o) n += v;
            }
            if (e < p.E) cum[e + 1] = carry + n;
            carry += __shfl_sync(kAll, n, 31);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    Ctl ctl;
    ctl.abort = &abort_flag;
    ctl.err = p.err;
    ctl.spin = false;
    ctl.pipe_polls = kMaxSpins;
    Sched sched;
    sched.tiles_f = (p.N + kTile - 1) / kTile;
    sched.total = (long long)cum[p.E] * sched.tiles_f;
    const int nk = (p.K + 255) / 256;
    constexpr int kChunksPerStage = MX ? 2 : 4;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0;  // stages filled
            bool ok = true;
            for (long long id = blockIdx.x; ok && id < sched.total; id += gridDim.x) {
                const Tile t = tile_of(id, sched, start, cum, p.E);
                const int boxes = (t.rows + kBoxRows - 1) / kBoxRows;
                const uint8_t *sw = p.w_scales + ((long long)t.e * sched.tiles_f + t.f) * p.chunks * 512;
                const uint8_t *sa = p.a_scales + (long long)t.stile * p.chunks * 512;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % kStagesP;
                    if (!wait_phase<false, kPipe>(empty + 8 * s, ((it / kStagesP) & 1u) ^ 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = base + s * kStageBytes, bar = full + 8 * s;
                    const int c0 = k * kChunksPerStage;
                    const uint32_t sbytes = (uint32_t)min(kChunksPerStage, p.chunks - c0) * 512u;
                    mbar_arrive_expect_tx(bar, (uint32_t)(kTile + boxes * kBoxRows) * kTileBytes + 2 * sbytes);
                    tma_2d(at, &map_w, k * kTileBytes, t.e * p.N + t.f * kTile, bar);
                    for (int b = 0; b < boxes; ++b)
                        tma_2d(at + kOffB + b * kBoxRows * kTileBytes, &map_a, k * kTileBytes, t.row0 + b * kBoxRows, bar);
                    bulk_g2s(at + kOffSA, sw + (long long)c0 * 512, sbytes, bar);
                    bulk_g2s(at + kOffSB, sa + (long long)c0 * 512, sbytes, bar);
                }
            }
            // no copy may be in flight into a CTA that leaves
            for (uint32_t i = it > kStagesP ? it - kStagesP : 0; i < it; ++i)
                wait_phase<false, kDrain>(full + 8 * (i % kStagesP), (i / kStagesP) & 1u, ctl);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (long long id = blockIdx.x; ok && id < sched.total; id += gridDim.x, ++n) {
                const Tile t = tile_of(id, sched, start, cum, p.E);
                const uint32_t buf = n & 1u;
                if (!wait_phase<false, kPipe>(acc_empty + 8 * buf, ((n >> 1) & 1u) ^ 1u, ctl)) break;
                fence_after();
                const uint32_t columns = (uint32_t)(t.rows + 15) / 16 * 16;
                // E2M1 operands, both with K along the row; E8M0 scales for MXFP4; N / 8, M / 16
                const uint32_t idesc = (1u << 7) | (1u << 10) | ((columns >> 3) << 17) | ((MX ? 1u : 0u) << 23) |
                                       ((kTile >> 4) << 24);
                const uint32_t d = tmem + buf * kTile;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % kStagesP;
                    if (!wait_phase<false, kPipe>(full + 8 * s, (it / kStagesP) & 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t at = base + s * kStageBytes;
                    const uint32_t sa = tmem + kScaleColumn + (it & 1u) * 32u, sb = sa + 16u;
                    const uint64_t da = codes_desc(at), db = codes_desc(at + kOffB);
                    const uint64_t dsa = scales_desc(at + kOffSA), dsb = scales_desc(at + kOffSB);
                    auto scales = [&](int c) {
                        copy_scales(sa + 4 * c, dsa + 32 * c);
                        copy_scales(sb + 4 * c, dsb + 32 * c);
                    };
                    auto step = [&](int j) {
                        const uint32_t col = MX ? 4 * (j >> 1) : 4 * j;
                        const uint32_t half = MX ? (j & 1u) * 2u : 0u;  // which 2 of the 4 scale bytes
                        product<MX>(d, da + 2 * j, db + 2 * j, idesc | (half << 4) | (half << 29), sa + col, sb + col,
                                    k > 0 || j > 0);
                    };
                    if (k * 256 + 256 <= p.K) {  // unrolled: the issuing thread sets the pace
#pragma unroll
                        for (int c = 0; c < kChunksPerStage; ++c) scales(c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) step(j);
                    } else {
                        const int nc = p.chunks - k * kChunksPerStage, steps = (p.K - k * 256 + 63) / 64;
                        for (int c = 0; c < nc; ++c) scales(c);
                        for (int j = 0; j < steps; ++j) step(j);
                    }
                    commit(empty + 8 * s);
                }
                if (ok) commit(acc_full + 8 * buf);
            }
            commit(done);  // every product has ended before tensor memory is freed
            wait_phase<false, kDrain>(done, 0, ctl);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;  // the lanes of tensor memory that this warp reads
        uint32_t n = 0;
        for (long long id = blockIdx.x; id < sched.total; id += gridDim.x, ++n) {
            const Tile t = tile_of(id, sched, start, cum, p.E);
            const uint32_t buf = n & 1u;
            if (!wait_phase<false, kPipe>(acc_full + 8 * buf, (n >> 1) & 1u, ctl)) break;
            fence_after();
            const int f = t.f * kTile + quad * 32 + lane;
            const bool odd = lane & 1;
            uint16_t *out = p.out + (long long)(t.row0 + odd) * p.N + (f & ~1);
            for (int c = 0; c < t.rows; c += 16) {
                uint32_t v[16];
                read16(tmem + ((uint32_t)(quad * 32) << 16) + buf * kTile + c, v);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    // lane pairs trade: the even lane stores two features of row c + i, the odd one of the next
                    const float x = __uint_as_float(v[i]) * p.alpha, y = __uint_as_float(v[i + 1]) * p.alpha;
                    const float got = __shfl_xor_sync(kAll, odd ? x : y, 1);
                    const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(got, y) : __floats2bfloat162_rn(x, got);
                    if (c + i + odd < t.rows && f < p.N)
                        *reinterpret_cast<__nv_bfloat162 *>(out + (long long)(c + i) * p.N) = h;
                }
            }
            fence_before();
            mbar_arrive(acc_empty + 8 * buf);
        }
        // rows of no group
        const long long first = (long long)start[p.E] * p.N / 8, last = (long long)p.M * p.N / 8;
        for (long long i = first + (long long)blockIdx.x * 128 + (threadIdx.x - 64); i < last;
             i += (long long)gridDim.x * 128)
            reinterpret_cast<uint4 *>(p.out)[i] = make_uint4(0, 0, 0, 0);
    }
    fence_before();
    __syncthreads();
    if (warp == 2) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns));
    }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn g_encode;
cudaError_t g_encode_status = cudaErrorUnknown;
std::once_flag g_encode_once;

// rows of `bytes` bytes, boxes of `box` rows by 128 bytes
cudaError_t make_map(CUtensorMap *map, const uint8_t *data, long long rows, long long bytes, int box)
{
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t boxes[2] = {(cuuint32_t)kTileBytes, (cuuint32_t)box}, ones[2] = {1, 1};
    const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(data), dims, strides, boxes,
                                ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_product(const ProductArgs &p, const uint8_t *a, const uint8_t *w, int fmt, int sms, bool pdl,
                           cudaStream_t st)
{
    std::call_once(g_encode_once, []() {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        g_encode_status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (g_encode_status == cudaSuccess && (q != cudaDriverEntryPointSuccess || !fn))
            g_encode_status = cudaErrorNotSupported;
        g_encode = reinterpret_cast<EncodeFn>(fn);
    });
    if (g_encode_status != cudaSuccess) return g_encode_status;
    CUtensorMap map_a, map_w;
    cudaError_t e = make_map(&map_a, a, p.M, p.K / 2, kBoxRows);
    if (e == cudaSuccess) e = make_map(&map_w, w, (long long)p.E * p.N, p.K / 2, kTile);
    if (e != cudaSuccess) return e;
    const size_t smem = 1024 + (size_t)kStagesP * kStageBytes + 2 * sizeof(int) * (size_t)(p.E + 1);
    auto *k = fmt ? product_kernel<true> : product_kernel<false>;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long row_tiles = (long long)p.M / kTile + (p.E < p.M ? p.E : p.M);
    const long long most = row_tiles * ((p.N + kTile - 1) / kTile);
    const int grid = (int)(most < sms ? most : sms);
    return launch_kernel(k, dim3((unsigned)grid), dim3(kThreads), smem, pdl, 1, st, map_a, map_w, p);
}

}  // namespace bn
