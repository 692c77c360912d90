// bn_product8.cu -- the experts' product of 8-bit integer rows and weights.
//
// For the rows m of group e (offsets[e] <= m < offsets[e + 1]) and n in [0, N):
//   out[m, n] = bf16(alpha * a_scale[m] * w_scale[e, n] * sum_k a[m, k] * w[e, n, k])
// with the sum exact.  Rows of no group are written as zeros.
//
// The device's 8-bit integer products are slower than its 16-bit ones by far, and
// whole numbers up to 2048 are exact in FP16, so codes are widened to FP16 on the
// way to the tensor core: a product of two is at most 2^14, and 1024 of them sum
// exactly in its FP32 accumulator.  After every 1024 the output warps add the
// accumulator to 32-bit integers in registers, while the other accumulator is filled.
//
// Weights are the tensor core's M operand.  They come to shared memory as codes (TMA,
// 128-byte swizzle, 128 values of K a stage); eight warps widen them, a lane a weight
// row, every second stage, into tensor memory, from where the tensor core takes its M
// operand: so they pass through shared memory as bytes only.
//
// Two shapes.  Narrow: one CTA, tiles of 128 features by 32 rows, whose codes two more warps
// widen into shared memory; where tiles are too few for the device, clusters of CTAs each
// sum a part of K.  Pairs of CTAs (cta_group::2): tiles of 256 by 128, of which each CTA
// loads half of either operand; rows are widened once by a kernel ahead into a workspace,
// as every feature tile reads them again.
//
// Measured.  Few rows: the stream of weights; 100 tokens with 8 of 256 experts of 6144 x
// 1024 (1.17 GB reached) 172 us, 6.8 TB/s; one token with 10 of 1024 x 8192 (84 MB) 22.6 us, of
// which the first codes take 2.3 to arrive.  Rings: with one ring for codes and products 28
// us, with the rows widened ahead 26; with 16 widening warps no faster.  Large groups: 4096
// tokens with 8 of 64, 4096 x 5120: 922 us alone, 1.49 PFLOP/s, 964 back to back; without the widening stores 11 % less
// time, with one product in eight 16 % less, with neither 20 %: the copies' 64 bytes a
// cycle and SM (60 is what one takes in), which wider tiles would lower, but 256 sums a
// lane pair do not fit the registers beside the widening warps.
#include <cuda_fp16.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"
#include "bn_tensor.cuh"

namespace bn {

namespace {

constexpr int kHalf = 128;       // features that one CTA loads for a tile
constexpr int kDepth = 128;      // values of K of a stage
constexpr int kExact = 8;        // stages whose sum is exact in FP32: 1024 products of at most 2^14
constexpr int kTmemColumns = 512;
constexpr int kAColumns = kDepth / 2;  // tensor memory columns of a stage's weights

template <bool PAIR>
struct Shape8 {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kTile = PAIR ? 256 : 128;   // features of an output tile
    static constexpr int kRows = PAIR ? 128 : 32;    // its rows
    static constexpr int kStep = PAIR ? 32 : 16;     // rows of a product are rounded up to this
    // Rings of their own: codes wait for copies from DRAM and are free once widened; rows, and
    // the weights in tensor memory, once the products have read them.
    static constexpr int kW = PAIR ? 8 : 7;          // stages of codes
    static constexpr int kX = PAIR ? 4 : 6;          // stages of rows, and of weights in tensor memory
    static constexpr int kWBytes = (kHalf + (PAIR ? 0 : kRows)) * kDepth;  // narrow: the rows' codes behind the weights'
    static constexpr int kAtom = kRows / kCtas * 128;  // rows of 64 values
    static constexpr int kBox = kRows / kCtas;       // rows of the larger box; the smaller one has half
    static constexpr int kXBytes = 2 * kAtom;
    static constexpr int kRingBytes = kW * kWBytes + kX * kXBytes;
    static constexpr int kColumnA = 2 * kRows;       // the weights in tensor memory, behind two accumulators
    static constexpr int kJoinBytes = PAIR ? 0 : (kRows + kMaxSplit) * kHalf * 4;
    static constexpr int kOutWarps = PAIR ? 8 : 4;
    static constexpr int kWideners = 8;              // warps that widen, two for every 32 weight rows
    static constexpr int kOutWarp = 4 + kWideners;   // warps: codes, products, 2 for rows, widening, output
    static constexpr int kThreads = 32 * (kOutWarp + kOutWarps);
    static constexpr size_t smem(int E) { return 1024 + (size_t)kRingBytes + kJoinBytes + 2 * sizeof(int) * (size_t)(E + 1); }
};
static_assert(Shape8<true>::kColumnA + Shape8<true>::kX * kAColumns <= kTmemColumns, "tensor memory");
static_assert(Shape8<false>::kColumnA + Shape8<false>::kX * kAColumns <= kTmemColumns, "tensor memory");

struct Maps8 {
    CUtensorMap w;           // codes: boxes of 128 rows by 128
    CUtensorMap x, x_small;  // rows, all of a tile's share or half: widened in boxes of 64 values (pairs), or codes of 128
};

// The product with its M operand in tensor memory.
template <bool PAIR>
__device__ __forceinline__ void product8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                     "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                     "r"((uint32_t)accumulate) : "memory");
}

// Four codes as FP16: c + 128 in the low bits of 1024 is 1152 + c, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342), k = 0x64806480u;
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&k));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), *reinterpret_cast<const __half2 *>(&k));
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// A place in a ring of N stages, and the parity of its round.
template <int N>
struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == N) {
            at = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ void store32(uint32_t tmem, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(tmem), "r"(v[0]), "r"(v[1]),
        "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool PAIR>
__global__ void __launch_bounds__(Shape8<PAIR>::kThreads, 1)
product8_kernel(const __grid_constant__ Maps8 maps, const __grid_constant__ Product8Args p)
{
    using S = Shape8<PAIR>;
    constexpr int kW = S::kW, kX = S::kX, kTile = S::kTile, kRows = S::kRows;
    constexpr int kSums = kRows / S::kCtas;  // columns of an output warp: all, or half of a pair's 128
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * kW + 2 * kX + 7];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    int *parts = reinterpret_cast<int *>(raw + (base - smem_addr(raw)) + S::kRingBytes);
    int *start = parts + S::kJoinBytes / 4;
    int *cum = start + p.E + 1;
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // w_full: this CTA's codes have landed; w_empty: they are widened; ready: a stage's
    // weights are in tensor memory and its rows in shared memory (a pair's on the first CTA's
    // barrier); empty: the products have read both
    const uint32_t w_full = smem_addr(bars), w_empty = w_full + 8 * kW, ready = w_empty + 8 * kW, empty = ready + 8 * kX;
    const uint32_t acc_full = empty + 8 * kX, acc_empty = acc_full + 16, done = acc_empty + 16, joined = done + 8, joinable = joined + 8;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const uint32_t parts_n = PAIR ? 1u : (uint32_t)p.split, part = PAIR || parts_n == 1 ? 0u : cluster_ctarank();
    const int ctas = PAIR ? 2 : p.split;
    const int unit = (int)blockIdx.x / ctas, units = (int)gridDim.x / ctas;

    griddep_launch_dependents();
    if (warp == 1 && elect_one()) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.x) : "memory");
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kW; ++i) {
            mbar_init(w_full + 8 * i, 1);
            mbar_init(w_empty + 8 * i, PAIR ? 4 : 5);
        }
        for (int i = 0; i < kX; ++i) {
            mbar_init(ready + 8 * i, S::kCtas * 4 + 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, S::kCtas * S::kOutWarps);
        }
        mbar_init(done, 1);
        mbar_init(joined, 1);
        mbar_init(joinable, parts_n * S::kOutWarps);
        fence_mbarrier_init();
    }
    if (warp == 3) tmem_alloc<PAIR>(smem_addr(&tmem_slot), kTmemColumns);
    __syncwarp();
    if (PAIR || parts_n > 1) cluster_arrive();  // this CTA's barriers are ready
    griddep_wait();
    group_tiles<kRows>(p.offsets, p.M, p.E, S::kThreads, start, cum, p.err);
    fence_before();
    __syncthreads();
    if (PAIR || parts_n > 1) cluster_wait();  // and the other CTAs'
    fence_after();
    const uint32_t tmem = tmem_slot;

    Ctl ctl;
    ctl.abort = &abort_flag;
    ctl.err = p.err;
    ctl.spin = false;
    ctl.pipe_polls = kMaxSpins;
    Tiles<kRows, PAIR ? S::kStep : 0> tiles(start, cum, p.E, (unsigned)((p.N + kTile - 1) / kTile), (unsigned)unit, (unsigned)units);
    Tile t = {};
    const uint32_t nk = (uint32_t)(p.K + kDepth - 1) / kDepth;
    // the stages of the sum that this CTA takes
    const int k0 = (int)(part * nk / parts_n), k1 = (int)((part + 1) * nk / parts_n);

    const uint32_t rows_at = base + kW * S::kWBytes;
    if (warp == 0) {  // the codes
        uint32_t it = 0;  // stages filled
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const int f0 = t.f * kTile + (int)rank * kHalf;
            for (int k = k0; k < k1; ++k, ++it) {
                const uint32_t s = it % kW;
                ok = __all_sync(kAll, wait_phase<false, kPipe>(w_empty + 8 * s, ((it / kW) & 1u) ^ 1u, ctl));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t at = base + s * S::kWBytes, bar = w_full + 8 * s;
                    const int rows = PAIR ? 0 : t.rows <= S::kBox / 2 ? S::kBox / 2 : S::kBox;
                    mbar_arrive_expect_tx(bar, (uint32_t)(kHalf + rows) * kDepth);
                    tma_3d<false>(at, &maps.w, k * kDepth, f0, t.e, bar);
                    if (!PAIR) tma_2d<false>(at + kHalf * kDepth, rows == S::kBox ? &maps.x : &maps.x_small, k * kDepth, t.row0, bar);
                }
            }
        }
        // no copy may be in flight into a CTA that leaves
        for (uint32_t i = it > kW ? it - kW : 0; i < it; ++i) wait_phase<false, kDrain>(w_full + 8 * (i % kW), (i / kW) & 1u, ctl);
        __syncwarp();
    } else if (PAIR && warp == 2) {  // the rows, widened by the kernel ahead
        Ring<kX> ring;
        uint32_t it = 0;  // stages filled
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const int columns = (t.rows + S::kStep - 1) / S::kStep * S::kStep;
            const int nb = columns / 2, b0 = t.row0 + (int)rank * nb;  // this CTA's half
            const bool small = nb <= S::kBox / 2;
            const uint32_t bytes = 2u * 128u * (small ? S::kBox / 2 : S::kBox);
            for (int k = k0; k < k1; ++k, ++it, ring.next()) {
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(empty + 8 * ring.at, ring.phase ^ 1u, ctl));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t x = rows_at + ring.at * S::kXBytes, bar = mapa(ready + 8 * ring.at, 0);
                    if (rank == 0) mbar_arrive_expect_tx(ready + 8 * ring.at, S::kCtas * bytes);
                    const CUtensorMap *map = small ? &maps.x_small : &maps.x;
                    tma_2d<PAIR>(x, map, k * kDepth, b0, bar);
                    tma_2d<PAIR>(x + S::kAtom, map, k * kDepth + 64, b0, bar);  // past K: zeros
                }
            }
        }
        // no copy, and no arrival of a product, may be in flight into a CTA that leaves
        const uint32_t old = it > kX ? it - kX : 0;
        for (uint32_t i = old; ok && i < it; ++i)
            ok = wait_phase<PAIR, kPipe>(empty + 8 * (i % kX), (i / kX) & 1u, ctl);
        // after a timeout the copies' barrier may never complete: give them a while
        if (!ok) for (const long long t0 = clock64(); clock64() - t0 < (1 << 22);) {}
        __syncwarp();
    } else if (!PAIR && (warp == 2 || warp == 3)) {  // the rows' codes, widened: every second stage
        // a lane takes a row's 64 codes of one half of the stage (up to 16 rows), or both
        Ring<kX> ring;
        const uint32_t turn = (uint32_t)warp & 1u;
        uint32_t it = 0;
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            const bool few = t.rows <= 16;
            const int row = few ? lane & 15 : lane, first = few ? 4 * (lane >> 4) : 0, last = few ? first + 4 : 8;
            for (int k = k0; k < k1; ++k, ++it, ring.next()) {
                if ((it & 1u) != turn) continue;
                const uint32_t s = it % kW;
                ok = __all_sync(kAll, wait_phase<false, kPipe>(empty + 8 * ring.at, ring.phase ^ 1u, ctl)) &&
                     __all_sync(kAll, wait_phase<false, kPipe>(w_full + 8 * s, (it / kW) & 1u, ctl));
                if (!ok) break;
                const uint32_t from = base + s * S::kWBytes + kHalf * kDepth + (uint32_t)row * 128u;
                const uint32_t to = rows_at + ring.at * S::kXBytes + (uint32_t)row * 128u;
#pragma unroll 4
                for (int c = first; c < last; ++c) {  // 16 codes: two pieces of 16 bytes of a row's 128
                    const uint4 q = load_shared(from + ((c ^ (row & 7)) << 4));
                    uint4 a, b;
                    widen4(q.x, a.x, a.y);
                    widen4(q.y, a.z, a.w);
                    widen4(q.z, b.x, b.y);
                    widen4(q.w, b.z, b.w);
                    const uint32_t x = to + (c >> 2) * S::kAtom;
                    store_shared(x + (((2 * (c & 3)) ^ (row & 7)) << 4), a);
                    store_shared(x + (((2 * (c & 3) + 1) ^ (row & 7)) << 4), b);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(w_empty + 8 * s);
                    mbar_arrive(ready + 8 * ring.at);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // of a pair's CTAs the first issues the products
        if (rank == 0) {
            Ring<kX> ring;
            uint32_t n = 0;  // sums of up to kExact stages
            bool ok = true;
            while (ok && tiles.next(t, lane)) {
                const uint32_t columns = (uint32_t)((t.rows + S::kStep - 1) / S::kStep * S::kStep);
                // FP32 sums of FP16 operands with K along the row; N / 8, M / 16
                const uint32_t idesc = (1u << 4) | ((columns >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
                for (int c = k0; ok && c < k1; c += kExact, ++n) {
                    const uint32_t buf = n & 1u;
                    ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_empty + 8 * buf, ((n >> 1) & 1u) ^ 1u, ctl));
                    if (!ok) break;
                    const uint32_t acc = tmem + buf * kRows;
                    const int end = min(c + kExact, k1);
                    for (int k = c; k < end; ++k, ring.next()) {
                        ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(ready + 8 * ring.at, ring.phase, ctl));
                        if (!ok) break;
                        fence_after();
                        const uint32_t a = tmem + S::kColumnA + ring.at * kAColumns;
                        const uint64_t b = rows_desc(rows_at + ring.at * S::kXBytes);
                        if (elect_one()) {
                            const auto step = [&](int j) {  // 16 values: 8 columns, 32 bytes along a row
                                product8<PAIR>(acc, a + 8 * j, b + (j >> 2) * (S::kAtom >> 4) + (j & 3) * 2, idesc, k > c || j > 0);
                            };
                            if ((k + 1) * kDepth <= p.K) {  // unrolled: the issuing thread sets the pace
#pragma unroll
                                for (int j = 0; j < 8; ++j) step(j);
                            } else {
                                const int steps = (p.K - k * kDepth + 15) / 16;
                                for (int j = 0; j < steps; ++j) step(j);
                            }
                            commit<PAIR>(empty + 8 * ring.at);
                            if (k == end - 1) commit<PAIR>(acc_full + 8 * buf);
                        }
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
    } else if (warp >= 4 && warp < S::kOutWarp) {
        const int quad = warp & 3, row = quad * 32 + lane;  // this lane's weight row, and its lane of tensor memory
        const uint32_t turn = (uint32_t)(warp - 4) >> 2;  // every kTurns-th stage is this warp's
        constexpr uint32_t kTurns = S::kWideners / 4;
        Ring<kX> ring;
        uint32_t it = 0;
        bool ok = true;
        while (ok && tiles.next(t, lane)) {
            for (int k = k0; k < k1; ++k, ++it, ring.next()) {
                if (it % kTurns != turn) continue;
                const uint32_t s = it % kW;
                // the products have read what this place of tensor memory held
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(empty + 8 * ring.at, ring.phase ^ 1u, ctl)) &&
                     __all_sync(kAll, wait_phase<false, kPipe>(w_full + 8 * s, (it / kW) & 1u, ctl));
                if (!ok) break;
                fence_after();
                const uint32_t from = base + s * S::kWBytes + row * 128;
                const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + S::kColumnA + ring.at * kAColumns;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = load_shared(from + (((4 * h + i) ^ (row & 7)) << 4));
                    if (h == 1) {  // the codes are in registers
                        __syncwarp();
                        if (lane == 0) mbar_arrive(w_empty + 8 * s);
                    }
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        widen4(q[i].x, v[8 * i], v[8 * i + 1]);
                        widen4(q[i].y, v[8 * i + 2], v[8 * i + 3]);
                        widen4(q[i].z, v[8 * i + 4], v[8 * i + 5]);
                        widen4(q[i].w, v[8 * i + 6], v[8 * i + 7]);
                    }
                    store32(to + 32 * h, v);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) arrive_first(ready + 8 * ring.at);
                    else mbar_arrive(ready + 8 * ring.at);
                }
            }
        }
        __syncwarp();
    } else if (warp >= S::kOutWarp) {
        const int quad = warp & 3;                   // the lanes of tensor memory that this warp reads
        const int half = (warp - S::kOutWarp) >> 2;  // of a pair's columns
        uint32_t n = 0, tile = 0;
        bool ok = true;
        for (; ok && tiles.next(t, lane); ++tile) {
            const int columns = (t.rows + S::kStep - 1) / S::kStep * S::kStep;
            const int lo = half ? columns / 2 : 0, hi = half ? t.rows : min(PAIR ? columns / 2 : columns, t.rows);
            int sums[kSums];
#pragma unroll
            for (int i = 0; i < kSums; ++i) sums[i] = 0;
            for (int c = k0; c < k1; c += kExact, ++n) {
                const uint32_t buf = n & 1u;
                ok = __all_sync(kAll, wait_phase<PAIR, kPipe>(acc_full + 8 * buf, (n >> 1) & 1u, ctl));
                if (!ok) break;
                fence_after();
                const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + buf * kRows;
#pragma unroll
                for (int b = 0; b < kSums / 16; ++b) {
                    if (lo + 16 * b < hi) {
                        uint32_t v[16];
                        read16(acc + lo + 16 * b, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sums[16 * b + i] += __float2int_rn(__uint_as_float(v[i]));
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) arrive_first(acc_empty + 8 * buf);
                    else mbar_arrive(acc_empty + 8 * buf);
                }
            }
            if (!ok) break;
            const int f0 = t.f * kTile + (int)rank * kHalf + quad * 32, f = f0 + lane;
            const float ws = f < p.N ? p.alpha * __ldg(p.w_scales + (long long)t.e * p.N + f) : 0.0f;
            if (!PAIR && parts_n > 1) {
                // every CTA of the cluster finishes its share of the rows
                const int share = (columns + (int)parts_n - 1) / (int)parts_n;
                ok = __all_sync(kAll, wait_phase<true, kPipe>(joinable, (tile & 1u) ^ 1u, ctl));
                if (!ok) break;
                const int r0 = (int)part * share, r1 = min(r0 + share, t.rows);
                if (quad == 0 && lane == 0) mbar_arrive_expect_tx(joined, parts_n * (uint32_t)max(r1 - r0, 0) * 512u);
                const uint32_t mine = smem_addr(parts) + 4u * (uint32_t)(quad * 32 + lane) + part * (uint32_t)share * 512u;
                int owner = 0, at = 0;  // the CTA that takes a row, and the row's place there
                uint32_t to = mapa(mine, 0), bar = mapa(joined, 0);
#pragma unroll
                for (int r = 0; r < kSums; ++r) {
                    if (r < t.rows) send_cluster(to + (uint32_t)at * 512u, (uint32_t)sums[r], bar);
                    if (++at == share) {
                        at = 0;
                        owner = min(owner + 1, (int)parts_n - 1);
                        to = mapa(mine, (uint32_t)owner);
                        bar = mapa(joined, (uint32_t)owner);
                    }
                }
                ok = __all_sync(kAll, wait_phase<true, kPipe>(joined, tile & 1u, ctl));
                if (!ok) break;
                const int *from = parts + quad * 32 + lane;
                for (int r = r0; r < r1; ++r, from += 128) {
                    int sum = 0;
                    for (int i = 0; i < (int)parts_n; ++i) sum += from[i * share * 128];
                    const float as = __ldg(p.a_scales + t.row0 + r);
                    if (f < p.N) p.out[(long long)(t.row0 + r) * p.N + f] = (uint16_t)bf16_pair((float)sum * as * ws, 0.0f);
                }
                __syncwarp();
                if (lane < (int)parts_n) arrive_cluster(mapa(joinable, (uint32_t)lane));
                continue;
            }
            // the rows' scales, a lane's share of the columns
            float as[(kSums + 31) / 32];
#pragma unroll
            for (int i = 0; i < (kSums + 31) / 32; ++i) {
                const int c = lo + 32 * i + lane;
                as[i] = c < hi ? __ldg(p.a_scales + t.row0 + c) : 0.0f;
            }
            const int fs = f0 + (lane & ~7);
            uint16_t *out = p.out + (long long)(t.row0 + (lane & 7)) * p.N + fs;
#pragma unroll
            for (int b = 0; b < kSums / 8; ++b) {
                if (lo + 8 * b < hi) {
                    uint32_t packed[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int c = 8 * b + 2 * i + j;
                            v[j] = (float)sums[c] * __shfl_sync(kAll, as[c / 32], c & 31) * ws;
                        }
                        packed[i] = bf16_pair(v[0], v[1]);
                    }
                    const uint4 v = transpose8(packed, lane);
                    const int c = lo + 8 * b;
                    if (c + (lane & 7) < hi && fs < p.N) *reinterpret_cast<uint4 *>(out + (long long)c * p.N) = v;
                }
            }
        }
        // rows of no group: before the first, and past the last
        constexpr int kFirst = 32 * S::kOutWarp;
        const long long step = (long long)gridDim.x * (S::kThreads - kFirst);
        const auto zeros = [&](long long row, long long end) {
            const long long last = end * p.N / 8;
            for (long long i = row * p.N / 8 + (long long)blockIdx.x * (S::kThreads - kFirst) + (threadIdx.x - kFirst); i < last; i += step)
                reinterpret_cast<uint4 *>(p.out)[i] = make_uint4(0, 0, 0, 0);
        };
        zeros(0, start[0]);
        zeros(start[p.E], p.M);
    }
    fence_before();
    __syncthreads();
    if (PAIR || parts_n > 1) cluster_sync_all();  // the others' products, or parts, reach this CTA's shared memory
    if (warp == 3) {
        fence_after();
        tmem_free<PAIR>(tmem, kTmemColumns);
    }
}

// Codes as FP16, 16 a thread: 16 bytes in and 32 out, which memory bounds (8192 rows of
// 5120 from a cold cache in 26 us, 4.8 TB/s).
__global__ void __launch_bounds__(256) widen_kernel(const uint4 *codes, long long n, uint4 *out)
{
    griddep_launch_dependents();
    griddep_wait();
    const long long step = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const uint4 q = __ldg(codes + i);
        uint4 a, b;
        widen4(q.x, a.x, a.y);
        widen4(q.y, a.z, a.w);
        widen4(q.z, b.x, b.y);
        widen4(q.w, b.z, b.w);
        out[2 * i] = a;
        out[2 * i + 1] = b;
    }
}

template <bool PAIR>
cudaError_t launch_shape8(const Product8Args &p, const Maps8 &maps, int sms, bool pdl, cudaStream_t st)
{
    using S = Shape8<PAIR>;
    static KernelSetup setup;
    auto *k = product8_kernel<PAIR>;
    const cudaError_t e = setup(k, (int)S::smem(kMaxExperts));
    if (e != cudaSuccess) return e;
    const int ctas = PAIR ? 2 : p.split;
    const long long groups = p.E < p.M ? p.E : p.M;
    const long long most = ((long long)p.M + groups * (S::kRows - 1)) / S::kRows * ((p.N + S::kTile - 1) / S::kTile);
    const long long units = PAIR || ctas == 1 ? sms / ctas : resident_clusters(k, ctas, S::kThreads, S::smem(kMaxExperts), sms);
    const int grid = (int)(most < units ? most : units) * ctas;
    return launch_kernel(k, dim3((unsigned)grid), dim3(S::kThreads), S::smem(p.E), pdl, ctas, st, maps, p);
}

}  // namespace

// Which shape: pairs where that makes fewer rounds of tiles over the device (groups are taken to
// leave half a tile each).  Measured, narrow / pairs (us in a graph): 100 tokens with 8 of 256
// experts of 6144 x 1024 180 / 181 (as many rounds); 500 with 8 of 64, 2048 x 2048 102 / 63;
// 333 with 4 of 16, 1024 x 2048 26.7 / 19.6; 256 with 2 of 8, 4096 x 4096 59 / 37; 4096 with 8 of
// 64, 4096 x 5120 2869 / 938.  A narrow tile's sum is split as in bn_linear.cu; a join costs
// 5 stages of 128 values.
bool product8_pairs(const Product8Args &p, int sms, int *split)
{
    const long long groups = p.E < p.M ? p.E : p.M, nk = (p.K + kDepth - 1) / kDepth;
    const auto rounds = [&](int rows, int tile, int units) {
        const long long even = p.M / rows + groups / 2, n = even > groups ? even : groups;
        return (n * ((p.N + tile - 1) / tile) + units - 1) / units;
    };
    constexpr int kRows = Shape8<false>::kRows;
    const long long tiles = ((long long)p.M + groups * (kRows - 1)) / kRows * ((p.N + 127) / 128);
    *split = choose_split(tiles, nk, 5, (tiles + sms - 1) / sms * nk, sms);
    if (*split > 1 || p.M <= kRows) return false;
    return rounds(Shape8<true>::kRows, Shape8<true>::kTile, sms / 2) < rounds(kRows, 128, sms);
}

cudaError_t launch_product8(Product8Args p, const int8_t *w, void *workspace, int sms, bool pdl, cudaStream_t st)
{
    cudaError_t e = tensor_maps_ready();
    if (e != cudaSuccess) return e;
    Maps8 m;
    const bool pair = product8_pairs(p, sms, &p.split) && workspace;
    if (pair) {
        const long long n = (long long)p.M * p.K / 16, blocks = (n + 255) / 256, most = 16LL * sms;
        e = launch_kernel(widen_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, pdl, 1, st,
                          reinterpret_cast<const uint4 *>(p.a), n, static_cast<uint4 *>(workspace));
        if (e != cudaSuccess) return e;
    }
    const auto codes = [&](CUtensorMap *map, int box) {
        return make_map<2>(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.a, {(cuuint64_t)p.K, (cuuint64_t)p.M}, {kDepth, (cuuint32_t)box},
                           CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const auto widened = [&](CUtensorMap *map, int box) {
        return make_map<2>(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, workspace, {(cuuint64_t)p.K, (cuuint64_t)p.M}, {64, (cuuint32_t)box},
                           CU_TENSOR_MAP_SWIZZLE_128B);
    };
    e = make_map<3>(&m.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, {(cuuint64_t)p.K, (cuuint64_t)p.N, (cuuint64_t)p.E}, {kDepth, kHalf, 1},
                    CU_TENSOR_MAP_SWIZZLE_128B);
    const int box = pair ? Shape8<true>::kBox : Shape8<false>::kBox;
    if (e == cudaSuccess) e = pair ? widened(&m.x, box) : codes(&m.x, box);
    if (e == cudaSuccess) e = pair ? widened(&m.x_small, box / 2) : codes(&m.x_small, box / 2);
    if (e != cudaSuccess) return e;
    return pair ? launch_shape8<true>(p, m, sms, pdl, st) : launch_shape8<false>(p, m, sms, pdl, st);
}

}  // namespace bn
