// bn_tensor.cuh -- what the experts' products share: the walk over the output tiles
// of ragged groups, TMA and tensor-core instructions, the way of an accumulator to
// memory, and tensor maps on the host.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda.h>

#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {

using namespace dev;

namespace {

constexpr unsigned kAll = 0xffffffffu;

// One thread of a converged warp.  The product's and the copies' operands live in
// uniform registers; behind elect.sync the compiler knows that one thread runs.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// The groups' first rows (start) and the row tiles of TILE rows before each group
// (cum), E + 1 of either, in shared memory.  The caller synchronises its threads.  The
// first warp loads the offsets for itself, so that it waits for one load, not for a
// barrier after it (which took 2400 cycles of a call with 256 experts).
template <int TILE>
__device__ __forceinline__ void group_tiles(const int32_t *offsets, int M, int E, int threads, int *start, int *cum, unsigned *err)
{
    const auto offset = [&](int e) { return offsets ? __ldg(offsets + e) : e * M; };
    const auto inside = [&](int o) { return min(max(o, 0), M); };
    if (threadIdx.x < 32) {  // a lane takes its share of consecutive groups
        const int lane = threadIdx.x;
        const int share = (E + 31) / 32, e0 = min(lane * share, E), e1 = min(e0 + share, E);
        int n = 0, from = inside(offset(e0));
        bool falls = false;  // a falling offset: an empty group
#pragma unroll 8
        for (int e = e0; e < e1; ++e) {
            const int to = inside(offset(e + 1));
            cum[e] = n;
            n += (max(to - from, 0) + TILE - 1) / TILE;
            falls |= to < from;
            from = to;
        }
        if (falls) atomicOr(err, BN_DEVERR_OFFSETS);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) cum[E] = before;
        before -= n;
#pragma unroll 8
        for (int e = e0; e < e1; ++e) cum[e] += before;
    }
    for (int e = threadIdx.x; e <= E; e += threads) {
        const int o = offset(e);
        if (o < 0 || o > M) atomicOr(err, BN_DEVERR_OFFSETS);
        start[e] = inside(o);
    }
}

// The cluster's barrier in two halves: what its threads did before arriving is seen by all
// that have waited.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct Tile {
    int e, f, row0, rows, stile;
};

// The output tiles in order: experts one after another; of one expert, the row
// tiles of a feature tile next to each other, so that CTAs that run together
// share its weights in L2.  Every unit (a CTA or a pair) takes every step-th
// tile.  Called by whole warps: a warp keeps its place among the experts and the
// lanes look at the next 32 together, because the issuing warp has nothing in
// flight while it looks for its next tile.
// EVEN (pairs): a group's row tiles are alike, to EVEN rows, instead of whole ones and a rest.
// Where groups have two or four tiles, an even step gave some units whole tiles throughout
// and others rests (tensor pipe 33 to 90 % active over the SMs; 909 us, then 852).
template <int TILE, int EVEN = 0>
class Tiles {
public:
    __device__ Tiles(const int *start, const int *cum, int E, unsigned tiles_f, unsigned first, unsigned step)
        : start_(start), cum_(cum), E_(E), e_(0), tiles_f_(tiles_f), step_(step), id_(first),
          total_((unsigned long long)(unsigned)cum[E] * tiles_f)
    {
    }
    // The next tile, or false past the last one.
    __device__ __forceinline__ bool next(Tile &t, int lane)
    {
        if (id_ >= total_) return false;
        // row tiles before this tile: 32-bit arithmetic where the tile numbers fit
        const unsigned tt = total_ >> 32 ? (unsigned)(id_ / tiles_f_) : (unsigned)id_ / tiles_f_;
        unsigned past;
        do {  // experts that end at or before it
            const int e = e_ + 1 + lane;
            past = __popc(__ballot_sync(kAll, e <= E_ && (unsigned)cum_[min(e, E_)] <= tt));
            e_ += (int)past;
        } while (past == 32);
        const unsigned c = (unsigned)cum_[e_], nt = (unsigned)cum_[e_ + 1] - c;
        const unsigned local = (unsigned)(id_ - (unsigned long long)c * tiles_f_);
        const int s0 = start_[e_], s1 = start_[e_ + 1];
        t.e = e_;
        t.f = nt == 1 ? (int)local : (int)(local / nt);
        const int r = (int)(local - (unsigned)t.f * nt);
        const int height = EVEN ? (int)(((unsigned)(s1 - s0) + nt - 1) / nt + EVEN - 1) / max(EVEN, 1) * EVEN : TILE;
        t.row0 = s0 + r * height;
        t.rows = min(height, s1 - t.row0);
        t.stile = (s0 >> 7) + e_ + r * (TILE / 128);
        id_ += step_;
        return true;
    }

private:
    const int *start_, *cum_;
    int E_, e_;
    unsigned tiles_f_, step_;
    unsigned long long id_, total_;
};

// A box into this CTA's shared memory; its bytes count on `bar`, which for a
// pair is the first CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// The same of three dimensions.
template <bool PAIR>
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// Four rows of a map whose box is one row, one under the other; rows outside the map
// are zeros.
template <bool PAIR>
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *map, int x, int4 y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst), "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w),
            "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst), "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w),
            "r"(bar) : "memory");
}

// Shared-memory operand descriptor of rows of 128 bytes with K along them: 128-byte
// swizzle, 8 rows apart by 1024 bytes.
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

// Arrive on `bar` (of both CTAs of a pair) when every product so far has ended.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same on this CTA's barrier alone.
template <bool PAIR>
__device__ __forceinline__ void commit_here(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        commit<false>(bar);
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Arrive on a barrier of the pair's first CTA.  What it orders are reads of tensor
// memory, which the tcgen05 fences cover; a release at cluster scope would wait for
// the CTA's stores in flight (1350 cycles measured).
__device__ __forceinline__ void arrive_first(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapa(bar, 0)) : "memory");
}

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

// Each lane of eight holds eight rows of its own feature (two a word); after it,
// lane i holds the eight features of row i.
__device__ __forceinline__ uint4 transpose8(const uint32_t *w, int lane)
{
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl_xor_sync(kAll, w[i], 1);
        a[i] = lane & 1 ? __byte_perm(o, w[i], 0x7632) : __byte_perm(w[i], o, 0x5410);
    }
    uint32_t b[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t keep = lane & 2 ? a[2 * i + 1] : a[2 * i];
        const uint32_t o = __shfl_xor_sync(kAll, lane & 2 ? a[2 * i] : a[2 * i + 1], 2);
        b[i][0] = lane & 2 ? o : keep;
        b[i][1] = lane & 2 ? keep : o;
    }
    const uint32_t o0 = __shfl_xor_sync(kAll, lane & 4 ? b[0][0] : b[1][0], 4);
    const uint32_t o1 = __shfl_xor_sync(kAll, lane & 4 ? b[0][1] : b[1][1], 4);
    return lane & 4 ? make_uint4(o0, o1, b[1][0], b[1][1]) : make_uint4(b[0][0], b[0][1], o0, o1);
}

__device__ __forceinline__ uint4 load_shared(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store_shared(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A value into the shared memory of a CTA of the cluster, counted on its barrier there.
__device__ __forceinline__ void send_cluster(uint32_t addr, uint32_t v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

constexpr int kMaxSplit = 8;  // CTAs that share a tile's sum

// By how many CTAs to split the sums of `tiles` tiles of `stages` stages: rounds over the
// device times the stages of a part, a join of parts costing `join` stages more; 1 unless
// that saves a tenth of `whole`, the same count without a split.
inline int choose_split(long long tiles, long long stages, long long join, long long whole, int sms)
{
    int best = 1;
    long long least = whole * 9;
    for (int s = 2; s <= kMaxSplit && s * 4 <= stages; ++s) {
        const long long units = sms > s ? sms / s : 1, cost = (tiles + units - 1) / units * ((stages + s - 1) / s + join) * 10;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// Clusters of `split` CTAs that the device holds at once, looked up once per device.
template <typename... P>
int resident_clusters(void (*kernel)(P...), int split, int threads, size_t smem, int sms)
{
    static std::atomic<int> known[64][kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return sms / split;
    const int at = split;
    int n = dev < 64 ? known[dev][at].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms / split * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)split;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = sms / split;
    }
    if (dev < 64) known[dev][at].store(n, std::memory_order_relaxed);
    return n;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn g_encode;
cudaError_t g_encode_status = cudaErrorUnknown;
std::once_flag g_encode_once;

// CUDA's encoder of tensor maps, looked up once.
cudaError_t tensor_maps_ready()
{
    std::call_once(g_encode_once, []() {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        g_encode_status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (g_encode_status == cudaSuccess && (q != cudaDriverEntryPointSuccess || !fn))
            g_encode_status = cudaErrorNotSupported;
        g_encode = reinterpret_cast<EncodeFn>(fn);
    });
    return g_encode_status;
}

// `dims` elements of `size` bytes in boxes, densely, or rows (the second dimension)
// `ld` elements apart.
template <int RANK>
cudaError_t make_map(CUtensorMap *map, CUtensorMapDataType type, int size, const void *data, const cuuint64_t (&dims)[RANK],
                     const cuuint32_t (&box)[RANK], CUtensorMapSwizzle swizzle, cuuint64_t ld = 0)
{
    cuuint64_t strides[RANK - 1], bytes = (cuuint64_t)size;
    cuuint32_t ones[RANK];
    for (int i = 0; i < RANK; ++i) {
        bytes *= i == 0 && ld ? ld : dims[i];
        if (i < RANK - 1) strides[i] = bytes;
        ones[i] = 1;
    }
    const CUresult r = g_encode(map, type, RANK, const_cast<void *>(data), dims, strides, box, ones,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

}  // namespace bn
