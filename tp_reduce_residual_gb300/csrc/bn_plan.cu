// bn_plan.cu -- the plan that groups token slots by expert.
//
// Slot i = t * k + j of ids goes to place
//   perm[i] = offsets[id_i] + number of slots i' < i with the same id,
// offsets[e] = number of slots of experts below e, and rows[perm[i]] = t: a
// stable counting sort, so every place is decided by the ids alone.  Slots
// without an expert (id -1) come after all groups, from place offsets[E] on.
//
// One launch, no scratch memory: a cluster of up to 16 CTAs splits the slots,
// each warp a run of them.  Every warp counts its run per expert in shared
// memory; a scan over the warps, the CTAs (their totals read through
// distributed shared memory) and the experts turns counts into places; a second
// pass over the run hands them out.  Within 32 slots __match_any_sync finds
// equal ids.  Latency bounds it (the bytes are a few hundred KB), so loads are
// issued several at a time: ids eight steps ahead, the other CTAs' totals together
// (131072 slots 14.1 us; one at a time 22).  610 slots take 3.9 us.
#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {
using namespace dev;

namespace {

constexpr unsigned kAll = 0xffffffffu;

constexpr int kThreads = 512;
constexpr int kMostCtas = 16;
constexpr int kAhead = 8;  // steps of 32 slots whose ids are loaded together

__device__ __forceinline__ unsigned ld_cluster(uint32_t addr)
{
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a, int per_warp)
{
    extern __shared__ unsigned smem[];
    const int nb = a.E + 1;                   // experts, and the slots without one
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned *count = smem;                   // [warps][nb]
    unsigned *total = count + warps * nb;     // [nb] this CTA's slots of each expert
    unsigned *base = total + nb;              // [nb] first place of this CTA's slots
    __shared__ unsigned sums[33];
    const uint32_t cta = cluster_ctarank(), ctas = cluster_nctarank();

    for (int i = threadIdx.x; i < warps * nb; i += blockDim.x) count[i] = 0;
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();

    // unsigned: a step past the last of almost 2^31 slots stays a number past it
    const unsigned long long first = ((unsigned long long)cta * warps + warp) * (unsigned)per_warp;
    const unsigned lo = (unsigned)min(first, (unsigned long long)a.slots);
    const unsigned hi = (unsigned)min(first + (unsigned)per_warp, (unsigned long long)a.slots);
    unsigned *mine = count + warp * nb;
    bool bad = false;
    int id[kAhead];
    const auto load = [&](unsigned i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const unsigned i = i0 + 32 * u + lane;
            id[u] = i < hi ? __ldg(a.ids + i) : -1;
        }
    };
    const auto bucket_of = [&](int v) { return (unsigned)v < (unsigned)a.E ? v : a.E; };
    for (unsigned i0 = lo; i0 < hi; i0 += 32 * kAhead) {  // counting needs no order
        load(i0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (i0 + 32 * u + lane < hi) {
                bad |= id[u] < -1 || id[u] >= a.E;
                atomicAdd(mine + bucket_of(id[u]), 1u);
            }
    }
    if (bad) atomicOr(a.err, BN_DEVERR_EXPERT_RANGE);
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += blockDim.x) {
        unsigned run = 0;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const unsigned c = count[w * nb + b];
            count[w * nb + b] = run;
            run += c;
        }
        total[b] = run;
    }
    cluster_sync_all();
    // experts in chunks of one per thread, with a carry between chunks
    unsigned carry = 0;
    for (int b0 = 0; b0 < nb; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        unsigned all = 0, before = 0;
        if (b < nb) {
            const uint32_t at = smem_addr(total + b);
            unsigned v[kMostCtas];
#pragma unroll
            for (uint32_t c = 0; c < kMostCtas; ++c) v[c] = c < ctas ? ld_cluster(mapa(at, c)) : 0u;
#pragma unroll
            for (uint32_t c = 0; c < kMostCtas; ++c) {
                before += c < cta ? v[c] : 0u;
                all += v[c];
            }
        }
        unsigned run = all;  // inclusive scan over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(kAll, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) sums[warp] = run;
        __syncthreads();
        if (warp == 0) {
            const unsigned own = lane < warps ? sums[lane] : 0u;
            unsigned s = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(kAll, s, o);
                if (lane >= o) s += v;
            }
            sums[lane] = s - own;
            if (lane == 31) sums[32] = s;
        }
        __syncthreads();
        const unsigned start = carry + sums[warp] + run - all;
        carry += sums[32];
        if (b < nb) {
            base[b] = start + before;
            if (cta == 0) a.offsets[b] = (int)start;
        }
        __syncthreads();
    }
    // hand out the places, in slot order
    const unsigned below = (1u << lane) - 1u;
    for (unsigned i0 = lo; i0 < hi; i0 += 32 * kAhead) {
        load(i0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const unsigned i = i0 + 32 * u + lane;
            if (i - lane >= hi) break;
            const int b = i < hi ? bucket_of(id[u]) : -1;
            const unsigned same = __match_any_sync(kAll, b);
            unsigned place = 0;
            if (b >= 0) place = base[b] + mine[b] + __popc(same & below);
            __syncwarp();
            if (b >= 0 && (same & below) == 0) mine[b] += __popc(same);
            __syncwarp();
            if (b >= 0) {
                a.rows[place] = (int)(i / (unsigned)a.k);
                for (int r = 0; r < a.R; ++r) a.perm[(long long)r * a.slots + i] = (int)place;
            }
        }
    }
    cluster_sync_all();  // no CTA leaves while its totals may be read
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, bool pdl, cudaStream_t st)
{
    // A slot a thread, up to 16 CTAs; then longer runs per warp.  CTAs of 1024 threads
    // take as long at 131072 slots (13.4 us against 13.6) and longer at 1528 (4.5, 3.5).
    constexpr int warps = kThreads / 32;
    int ctas = 1;
    while (ctas < kMostCtas && (long long)ctas * kThreads < a.slots) ctas *= 2;
    const long long share = ((long long)a.slots + ctas * warps - 1) / (ctas * warps);
    const int per_warp = (int)((share + 31) / 32 * 32);
    const auto smem = [](int E) { return sizeof(unsigned) * (size_t)(warps + 2) * (size_t)(E + 1); };
    static KernelSetup setup;
    const cudaError_t e = setup(plan_kernel, (int)smem(kMaxExperts), true);
    if (e != cudaSuccess) return e;
    return launch_kernel(plan_kernel, dim3((unsigned)ctas), dim3(kThreads), smem(a.E), pdl, ctas, st, a,
                         per_warp);
}

}  // namespace bn
