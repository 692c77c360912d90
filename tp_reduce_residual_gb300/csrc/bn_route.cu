// bn_route.cu -- routing of tokens to experts, and its gradient.
//
// Forward, for one token's logits x[0..E):
//   s_e = 1 / (1 + exp(-x_e))  or  exp(x_e - max x) / sum exp(x - max x)
//   key_e = s_e + bias_e; without a bias, and unless groups are ranked by a sum
//     of scores, key_e = x_e (the scores rise with the logits)
//   groups > 1: a group's rank is the sum of its `group_top` largest keys; the
//     `top_groups` groups of the highest rank stay
//   ids = the k largest keys left, equal keys by rising index
//   w   = scale * s_id, or scale * s_id / sum over the k of s; sigmoids over their
//     sum are taken as s exp(-m) = 1 / (exp(m) + exp(m - x)), m the largest chosen
//     logit but at most 0, so that small ones keep their digits
// A logit or bias of -inf takes its expert out; slots for which no expert is
// left get id -1 and weight 0.  A NaN logit or key takes its expert out and
// makes the row's weights NaN; so does a logit of inf a softmax's (inf - inf).
//
// The order of keys is decided as in exact arithmetic.  Logits of 16 bits compare
// exactly.  Sums s + bias are computed in 32 bits with a bound on their error, and
// keys give their lowest bits to an index (below); where two keys (or two groups'
// ranks) whose order matters differ by less than the bound, the choice is made
// again with 64-bit keys: among the few candidates if only the experts' order is
// open, else for the whole row.
//
// One warp per token: a lane holds VPT consecutive experts.  Each lane sorts its
// keys once (an odd-even merge sorting network; the position in the lane rides in
// the keys' lowest bits, so that a comparison is one instruction), then k rounds
// take the largest of the 32 heads (redux.sync) and advance one lane.  What bounds
// it is instruction issue: 1390 instructions a token at 256 experts in 8 groups with
// a bias and k = 8 (ncu).  16384 such tokens take 27 us (IPC 3.1; the bytes alone
// would take 1.4), one token 3.6.  Searching the lane's 8 keys again after each round,
// with indexes apart, took 47 us, 20 of them a tail of rows that were selected whole
// in 64 bits.
#include <cfloat>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {
using namespace dev;

namespace {

constexpr int kWarps = 4;           // tokens per block
constexpr unsigned kAll = 0xffffffffu;
constexpr int kNone = 0x7fffffff;

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_min(float v) { return -warp_max(-v); }
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Elements [lane * VPT, lane * VPT + VPT) of a row of n, `fill` past the end.
template <typename T, int VPT>
__device__ __forceinline__ void load_row(const T *row, int n, int lane, bool vec, float fill, float *x)
{
    constexpr int W = 16 / (int)sizeof(T);  // elements per 16-byte load
    if constexpr (VPT >= W) {
        if (vec) {
#pragma unroll
            for (int c = 0; c < VPT / W; ++c) {
                const int i = lane * VPT + c * W;
                union { uint4 q; T t[W]; } u;
                if (i < n) {  // n is a multiple of W
                    u.q = __ldg(reinterpret_cast<const uint4 *>(row + i));
#pragma unroll
                    for (int j = 0; j < W; ++j) x[c * W + j] = to_f32(u.t[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) x[c * W + j] = fill;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = lane * VPT + j;
        x[j] = i < n ? to_f32(row[i]) : fill;
    }
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ double sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

// Error bound of a 32-bit score: expf is within 2 units in the last place
// (2^-22 relative), the addition within 2^-24, rcp.approx within 2^-23: under
// 1.5 * 2^-22 of s <= 1 for the sigmoid.  The softmax's sum of at most 1024 terms
// (32 in a lane, 5 levels) adds 37 * 2^-24 and x - max its own rounding, at most
// max(d exp(-d)) * 2^-24: under 2^-18 of the largest probability together.
constexpr float kSigmoidError = 1.5f * 0x1p-22f;
constexpr float kSoftmaxError = 0x1p-18f;

// Where exp(-x) passes 64 bits, a sigmoid counts as 0: chosen logits that are all
// below it (masks of the type's lowest value) have no weights.
constexpr float kNoSigmoid = -709.7827f;

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---- 64-bit selection, for rows whose order 32 bits do not tell ------------------------

// Take the n largest of the warp's keys, one per round; lane j ends with the
// j-th id (-1 where nothing is left).
template <int VPT>
__device__ __forceinline__ int take64(double *key, int lane, int n)
{
    int id = -1;
    for (int r = 0; r < n; ++r) {
        double best = key[0];
        int bi = 0;
#pragma unroll
        for (int j = 1; j < VPT; ++j)
            if (key[j] > best) { best = key[j]; bi = j; }
        const double m = warp_max(best);
        if (!(m > -(double)INFINITY)) break;
        const int i = __reduce_min_sync(kAll, best == m ? lane * VPT + bi : kNone);
        if (lane == r) id = i;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (lane * VPT + j == i) key[j] = -INFINITY;
    }
    return id;
}

template <typename F>
__device__ __forceinline__ void push2(F v, F &a, F &b)
{
    if (v > a) { b = a; a = v; }
    else if (v > b) b = v;
}

// The groups that stay, as bits, from the two largest keys of group `lane` (lanes
// past the groups hold -inf).  `gap`: how far the lowest rank that stays is above
// the highest that goes (inf if none goes); `largest`: the largest sum of the sizes
// of the keys that rank a group.  In 32 bits it is inf for two keys of the type's
// lowest value: no bound then tells anything, and the ranks are taken in 64 bits.
template <typename F>
__device__ __forceinline__ unsigned keep_groups(F r1, F r2, int lane, const RouteArgs &a, F &gap, F &largest)
{
    F rank = -INFINITY;
    if (lane < a.groups && r1 > (F)-INFINITY) rank = a.group_top > 1 && r2 > (F)-INFINITY ? r1 + r2 : r1;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
        const F o = __shfl_sync(kAll, rank, g);
        ahead += (o > rank || (o == rank && g < lane)) ? 1 : 0;
    }
    const bool keep = lane < a.groups && ahead < a.top_groups;
    const F low = -warp_max(keep && rank > (F)-INFINITY ? -rank : (F)-INFINITY);
    const F high = warp_max(!keep && lane < a.groups ? rank : (F)-INFINITY);
    const F size1 = r1 > (F)-INFINITY ? (r1 < 0 ? -r1 : r1) : (F)0, size2 = r2 > (F)-INFINITY ? (r2 < 0 ? -r2 : r2) : (F)0;
    largest = warp_max(a.group_top > 1 ? size1 + size2 : size1);
    gap = high > (F)-INFINITY ? low - high : (F)INFINITY;
    return __ballot_sync(kAll, keep);
}

// The whole row; `slot` is the warp's shared memory for 32 * VPT keys.
template <typename T, int VPT, bool SUMS>
__device__ __noinline__ int select64(const T *row, const RouteArgs &a, int lane, double *slot)
{
    float x[VPT];
    load_row<T, VPT>(row, a.E, lane, a.vec, -INFINITY, x);
    double key[VPT];
    if (!SUMS) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) key[j] = x[j];
    } else if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) key[j] = sigmoid((double)x[j]);
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPT; ++j) m = fmaxf(m, x[j]);
        m = warp_max(m);
        double sum = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            key[j] = x[j] > -INFINITY ? exp((double)x[j] - (double)m) : 0.0;
            sum += key[j];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int j = 0; j < VPT; ++j) key[j] /= sum;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = lane * VPT + j;
        key[j] += a.bias && e < a.E ? (double)__ldg(a.bias + e) : 0.0;
        if (!(x[j] > -INFINITY) || !(key[j] > -(double)INFINITY)) key[j] = -INFINITY;
    }
    if (a.groups > 1) {
        const int size = a.E / a.groups;
#pragma unroll
        for (int j = 0; j < VPT; ++j) slot[lane * VPT + j] = key[j];
        __syncwarp();
        double r1 = -INFINITY, r2 = -INFINITY, gap, largest;
        if (lane < a.groups)
            for (int i = 0; i < size; ++i) push2(slot[lane * size + i], r1, r2);
        const unsigned kept = keep_groups(r1, r2, lane, a, gap, largest);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = lane * VPT + j;
            if (e < a.E && !((kept >> (e / size)) & 1u)) key[j] = -INFINITY;
        }
    }
    return take64<VPT>(key, lane, a.k);
}

// The softmax's sum over the row in 64 bits; `top` is the largest logit.
template <typename T, int VPT>
__device__ __noinline__ double sum64(const T *row, const RouteArgs &a, int lane, float top)
{
    float x[VPT];
    load_row<T, VPT>(row, a.E, lane, a.vec, -INFINITY, x);
    double sum = 0;
#pragma unroll 1
    for (int j = 0; j < VPT; ++j) sum += x[j] > -INFINITY ? exp((double)x[j] - (double)top) : 0.0;
    return warp_sum(sum);
}

// A chosen or candidate expert's key in 64 bits; `sum` as above, for the softmax.
template <typename T, bool SUMS>
__device__ __forceinline__ double key64(const T *row, const RouteArgs &a, int id, float top, double sum)
{
    const double x = (double)to_f32(row[id]);
    if (!SUMS) return x;
    return (a.sigmoid ? sigmoid(x) : exp(x - (double)top) / sum) + (a.bias ? (double)__ldg(a.bias + id) : 0.0);
}

// The groups that stay, by 64-bit ranks, from the row's 32-bit keys in `slot`: lane
// g takes the four largest of group g, each known to within `error`, and ranks the
// group by the best of their 64-bit keys.  False where more than four may count.
template <typename T, int VPT, bool SUMS>
__device__ __noinline__ bool groups64(const T *row, const RouteArgs &a, int lane, const float *slot, float error,
                                      float top, double sum, unsigned *kept)
{
    const int size = a.E / a.groups;
    float v[5];
    int e[4] = {-1, -1, -1, -1};
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = -INFINITY;
    if (lane < a.groups)
        for (int i = 0; i < size; ++i) {
            const int at = lane * size + i;
            float x = slot[at];
            int id = at;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (x > v[q]) {
                    const float tv = v[q];
                    const int te = e[q];
                    v[q] = x;
                    e[q] = id;
                    x = tv;
                    id = te;
                }
            v[4] = fmaxf(v[4], x);
        }
    const float need = a.group_top > 1 ? v[1] : v[0];  // a key this far below cannot count
    // With at most four keys they are all there, whatever the error (it may be inf);
    // past this, e[0..3] are experts.
    bool ok = !(v[4] > -INFINITY) || need - v[4] > error;
    if (!ok) {
        // Keys that equal both the third and the fourth (ties: same logit, same bias) add nothing to the four.
        const float x3 = to_f32(row[e[3]]), b3 = a.bias ? __ldg(a.bias + e[3]) : 0.0f;
        ok = to_f32(row[e[2]]) == x3 && (!a.bias || __ldg(a.bias + e[2]) == b3);
        for (int i = 0; ok && i < size; ++i) {
            const int at = lane * size + i;
            if (slot[at] > -INFINITY && need - slot[at] <= error && at != e[0] && at != e[1])
                ok = to_f32(row[at]) == x3 && (!a.bias || __ldg(a.bias + at) == b3);
        }
    }
    double r1 = -INFINITY, r2 = -INFINITY, gap, largest;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (e[q] >= 0) push2(key64<T, SUMS>(row, a, e[q], top, sum), r1, r2);
    *kept = keep_groups(r1, r2, lane, a, gap, largest);
    return __all_sync(kAll, ok);
}

// The candidates, lane j < n the one of id `id`: lane j < k gets the j-th of them.
template <typename T, bool SUMS>
__device__ __noinline__ int order64(const T *row, const RouteArgs &a, int lane, int n, int id, float top, double sum,
                                    int *list)
{
    double key = -INFINITY;
    if (lane < n) key = key64<T, SUMS>(row, a, id, top, sum);
    int ahead = 0;
    for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(kAll, key, j);
        const int oid = __shfl_sync(kAll, id, j);
        ahead += (o > key || (o == key && oid < id)) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) list[ahead] = id;
    __syncwarp();
    return list[lane];
}

// ---- keys with an index in their lowest bits -----------------------------------------------

// Falling values of lane-local keys; of keys equal but for these bits the lower
// position comes first.
template <int VPT>
__device__ __forceinline__ float with_position(float v, int j)
{
    const uint32_t u = __float_as_uint(v), mask = VPT - 1, negative = (uint32_t)((int)u >> 31);
    return __uint_as_float((u & ~mask) | ((negative ^ (mask - j)) & mask));
}
template <int VPT>
__device__ __forceinline__ int position_of(float v)
{
    const uint32_t u = __float_as_uint(v), mask = VPT - 1, negative = (uint32_t)((int)u >> 31);
    return (int)((u ^ ~negative) & mask);
}
// What two keys are compared by.
template <int VPT>
__device__ __forceinline__ float without_position(float v)
{
    return __uint_as_float(__float_as_uint(v) & ~(uint32_t)(VPT - 1));  // -inf stays
}

// Batcher's odd-even merge sort, falling.
template <int VPT>
__device__ __forceinline__ void sort_keys(float *v)
{
#pragma unroll
    for (int p = 1; p < VPT; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < VPT; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < VPT && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const float hi = fmaxf(v[i + j], v[i + j + q]), lo = fminf(v[i + j], v[i + j + q]);
                        v[i + j] = hi;
                        v[i + j + q] = lo;
                    }
}

// SUMS: the keys are s + bias (or group ranks are sums of scores), else logits.
template <typename T, int VPT, bool SUMS>
__global__ void __launch_bounds__(kWarps * 32, VPT <= 8 ? 10 : 1) route_kernel(const __grid_constant__ RouteArgs a)
{
    __shared__ double slots[kWarps][32 * VPT];
    __shared__ int lists[kWarps][32];
    // 16-bit logits leave their low bits free: nothing is lost to the positions
    constexpr bool kExact = !SUMS && sizeof(T) == 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    griddep_launch_dependents();
    griddep_wait();
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (long long)t * a.ld;
    int *list = lists[warp];

    float key[VPT];
    load_row<T, VPT>(row, a.E, lane, a.vec, -INFINITY, key);
    bool nan = false;
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) nan |= key[j] != key[j];
    // softmax statistics, where a score depends on the whole row
    float inv = 0.0f;
    if (!a.sigmoid && (SUMS || !a.renormalize)) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) top = fmaxf(top, key[j]);  // a NaN is passed over
        top = warp_max(top);
        nan |= top == INFINITY;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) sum += key[j] > -INFINITY ? expf(key[j] - top) : 0.0f;
        sum = warp_sum(sum);
        inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // 0: every expert is masked
    }
    float serr = 0.0f;
    if constexpr (SUMS) {
        serr = a.sigmoid ? kSigmoidError : kSoftmaxError * inv;
        float b[VPT];
        if (a.bias)
            load_row<float, VPT>(a.bias, a.E, lane, a.bias_vec, 0.0f, b);
        else
#pragma unroll
            for (int j = 0; j < VPT; ++j) b[j] = 0.0f;
        float v[VPT];
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) v[j] = rcp_approx(1.0f + expf(-key[j])) + b[j];
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) v[j] = expf(key[j] - top) * inv + b[j];
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const bool in = key[j] > -INFINITY;
            nan |= in && v[j] != v[j];
            key[j] = in ? v[j] : -INFINITY;
        }
    }
    nan = __any_sync(kAll, nan);
#pragma unroll
    for (int j = 0; j < VPT; ++j)  // + 0 makes -0 a 0: they are equal
        key[j] = key[j] > -INFINITY ? with_position<VPT>(fminf(key[j], FLT_MAX) + 0.0f, j) : -INFINITY;

    // How far the difference of two keys may be off: their scores' errors, the
    // roundings of the sums with the bias, and the lowest bits of one (they are cut
    // off, so the two errors have one sign).
    const auto bound = [&](float v) { return 2.0f * serr + (VPT + 1) * 0x1p-23f * v + 0x1p-120f; };
    bool sure = true;  // of the groups that stay
    double all = 0.0;  // the softmax's sum in 64 bits, once it is wanted
    const auto sum_once = [&]() {
        if (SUMS && !a.sigmoid && all == 0.0) all = sum64<T, VPT>(row, a, lane, top);
        return all;
    };
    float *slot = reinterpret_cast<float *>(slots[warp]);
    const int size = a.E / a.groups, lanes = size / VPT;
    const bool whole = size % VPT == 0 && (lanes & (lanes - 1)) == 0;  // a group is so many whole lanes
    // of two ranks: twice as many keys, and a rounded sum each
    const auto uncertain = [&](float gap, float largest) {
        return !kExact && !(gap > 2.0f * bound(largest) + 0x1p-23f * largest);
    };
    if (a.groups > 1 && !whole) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) slot[lane * VPT + j] = without_position<VPT>(key[j]);
        __syncwarp();
        float r1 = -INFINITY, r2 = -INFINITY, gap, largest;
        if (lane < a.groups)
            for (int i = 0; i < size; ++i) push2(slot[lane * size + i], r1, r2);
        unsigned kept = keep_groups(r1, r2, lane, a, gap, largest);
        if constexpr (!kExact)
            if (uncertain(gap, largest))
                sure = groups64<T, VPT, SUMS>(row, a, lane, slot, bound(largest), top, sum_once(), &kept);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = lane * VPT + j;
            if (e < a.E && !((kept >> (e / size)) & 1u)) key[j] = -INFINITY;
        }
        __syncwarp();
    }
    sort_keys<VPT>(key);
    float head = without_position<VPT>(key[0]);
    if (a.groups > 1 && whole) {
        float p = head, q = VPT > 1 ? without_position<VPT>(key[VPT > 1 ? 1 : 0]) : -INFINITY, gap, largest;
        for (int o = 1; o < lanes; o <<= 1) {
            const float po = __shfl_xor_sync(kAll, p, o), qo = __shfl_xor_sync(kAll, q, o);
            q = fmaxf(fminf(p, po), fmaxf(q, qo));
            p = fmaxf(p, po);
        }
        const int src = min(lane * lanes, 31);
        unsigned kept = keep_groups(__shfl_sync(kAll, p, src), __shfl_sync(kAll, q, src), lane, a, gap, largest);
        if constexpr (!kExact)
            if (uncertain(gap, largest)) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) slot[lane * VPT + j] = -INFINITY;
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (key[j] > -INFINITY) slot[lane * VPT + position_of<VPT>(key[j])] = without_position<VPT>(key[j]);
                __syncwarp();
                sure = groups64<T, VPT, SUMS>(row, a, lane, slot, bound(largest), top, sum_once(), &kept);
                __syncwarp();
            }
        const int g = lane / lanes;
        if (g >= a.groups || !((kept >> g) & 1u)) head = -INFINITY;  // and so the lane's other keys
    }

    const unsigned own = 1u << lane, lanes_to = own | (own - 1u);  // this lane's bit, and those up to it
    int n = 0;             // chosen so far; lane j < n keeps the j-th key
    float at = -INFINITY;
    const auto choose = [&](float m) {  // m is the largest head: of equal ones the lowest lane's
        const unsigned best = __ballot_sync(kAll, head == m);
        if (lane == n) at = m;
        if ((best & lanes_to) == own) {
            list[n] = lane * VPT + position_of<VPT>(key[0]);
#pragma unroll
            for (int j = 0; j + 1 < VPT; ++j) key[j] = key[j + 1];
            key[VPT - 1] = -INFINITY;
            head = without_position<VPT>(key[0]);
        }
        ++n;
    };
    const int rounds = kExact ? a.k : a.k + 1;  // one more shows how far the last is from the next
    float m = -INFINITY;
    for (;;) {
        m = warp_max(head);
        if (m == -INFINITY || n == rounds) break;
        choose(m);
    }
    __syncwarp();
    int id = lane < n ? list[lane] : -1;
    if constexpr (!kExact) {
        // is the order of each and the next certain?
        const float x = id >= 0 ? to_f32(row[id]) : 0.0f, b = id >= 0 && a.bias ? __ldg(a.bias + id) : 0.0f;
        const float atn = __shfl_down_sync(kAll, at, 1), xn = __shfl_down_sync(kAll, x, 1),
                    bn = __shfl_down_sync(kAll, b, 1);
        // equal logits and biases have equal keys: the index decides
        const bool apart = at - atn > bound(fmaxf(fabsf(at), fabsf(atn))), same = x == xn && b == bn;
        bool open = __any_sync(kAll, lane + 1 < n && !(apart || same));
        const float last = __shfl_sync(kAll, at, a.k - 1);
        if (!open && __any_sync(kAll, lane == a.k - 1 && lane + 1 < n && !apart)) {
            // the last and the next are equal: is one of another key behind them within the bound?
            const float xl = __shfl_sync(kAll, x, a.k - 1), bl = __shfl_sync(kAll, b, a.k - 1);
            if (head > -INFINITY) {
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const float v = without_position<VPT>(key[j]);
                    if (v > -INFINITY && last - v <= bound(fmaxf(fabsf(last), fabsf(v)))) {
                        const int e = lane * VPT + position_of<VPT>(key[j]);
                        open |= to_f32(row[e]) != xl || (a.bias && __ldg(a.bias + e) != bl);
                    }
                }
            }
            open = __any_sync(kAll, open);
        }
        if (!sure || open) {
            // every expert that may belong among the k
            while (sure && n < 32 && m > -INFINITY && last - m <= bound(fmaxf(fabsf(last), fabsf(m)))) {
                choose(m);
                m = warp_max(head);
            }
            __syncwarp();
            if (!sure || n == 32) {
                id = select64<T, VPT, SUMS>(row, a, lane, slots[warp]);
                n = 32;  // its ids say how many there are
            } else
                id = order64<T, SUMS>(row, a, lane, n, lane < n ? list[lane] : -1, top, sum_once(), list);
        }
    }
    if (lane >= min(n, a.k)) id = -1;

    const bool on = lane < a.k && id >= 0;
    const float x = on ? to_f32(row[id]) : -INFINITY;
    float w, sum = 1.0f;
    if (a.sigmoid) {
        const float m = a.renormalize ? fminf(warp_max(x), 0.0f) : 0.0f;
        w = on && m > kNoSigmoid ? rcp_approx(expf(m) + expf(m - x)) : 0.0f;
        if (a.renormalize) sum = warp_sum(w);
    } else if (a.renormalize) {
        const float most = warp_max(x);
        nan |= most == INFINITY;
        w = on ? expf(x - most) : 0.0f;
        sum = warp_sum(w);
    } else {
        w = on ? expf(x - top) * inv : 0.0f;
    }
    if (lane < a.k) {
        w *= a.scale;
        if (a.renormalize) w /= fmaxf(sum, FLT_MIN);  // 0, or a half and more
        if (nan) w = NAN;
        const long long at_out = (long long)t * a.k + lane, shard = (long long)a.T * a.k;
        a.ids[at_out] = id;
        float *out = a.w + at_out;
        for (int r = 0; r < a.R; ++r, out += shard) *out = w;
    }
}

// Gradient of the weights with respect to the logits; the choice of experts
// (and with it the bias) has none.  With c = scale * sum over the shards of dw:
//   softmax, renormalised:  dx_j = w_j (c_j - sum_i w_i c_i),  w = softmax over the chosen
//   softmax:                dx_e = p_e (c_e - sum_j p_j c_j)   for every e (c_e = 0 unless chosen)
//   sigmoid:                dx_j = c_j s_j (1 - s_j)
//   sigmoid, renormalised:  dx_j = w_j (c_j - sum_i w_i c_i) (1 - s_j),  w = s / sum of s as in the forward
// 1 - s is computed as sigmoid(-x), which keeps its digits near s = 1.  A constant
// added to every c changes nothing but the plain sigmoid's gradient, so the c of an
// expert with more than a quarter of the weight is taken off first: its own
// c_j - sum_i w_i c_i is then a sum of the others' terms and not what is left of two
// equal numbers.  (With less weight nothing cancels, and to take it off would add an
// error of its size to all others.)  One warp per token: the chosen slots sit on lanes, are scattered into the warp's
// row in shared memory, and the row is written once with 16-byte stores.  16384
// tokens of 128 FP32 logits, dense: 6.1 us for 18 MB; 4096 of 256 BF16, sparse: 3.5.
template <typename T, int VPT, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(const __grid_constant__ RouteBackwardArgs a)
{
    __shared__ __align__(16) float rows[kWarps][32 * VPT];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    griddep_launch_dependents();
    griddep_wait();
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + (long long)t * a.ld;
    float *buf = rows[warp];
#pragma unroll
    for (int j = 0; j < VPT; ++j) buf[j * 32 + lane] = 0.0f;
    int id = -1;
    float c = 0.0f;
    if (lane < a.k) {
        const long long at = (long long)t * a.k + lane;
        id = a.ids[at];
        if (id < -1 || id >= a.E) {
            atomicOr(a.err, BN_DEVERR_EXPERT_RANGE);
            id = -1;
        }
        if (id >= 0) {
            for (int r = 0; r < a.R; ++r) c += a.dw[(long long)r * a.T * a.k + at];
            c *= a.scale;
        }
    }
    const bool on = id >= 0;
    const float x = on ? to_f32(row[id]) : -INFINITY;
    __syncwarp();
    float p[DENSE ? VPT : 1];
    int first = -1;  // the row's largest logit, if it was chosen and has much of the weight
    if constexpr (DENSE) {
        load_row<T, VPT>(row, a.E, lane, a.vec, -INFINITY, p);
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPT; ++j) top = fmaxf(top, p[j]);
        top = warp_max(top);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            p[j] = p[j] == -INFINITY ? 0.0f : expf(p[j] - top);  // NaN stays
            sum += p[j];
        }
        sum = warp_sum(sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int j = 0; j < VPT; ++j) p[j] *= inv;
        if (on) atomicAdd(buf + id, c);
        const unsigned best = __ballot_sync(kAll, on && x == top && inv > 0.25f);  // its p is inv
        if (best) first = __shfl_sync(kAll, id, __ffs(best) - 1);
    } else {
        const auto less_heaviest = [&](float w) {  // c less that of an expert of much weight
            const unsigned heavy = __ballot_sync(kAll, w > 0.25f);
            return heavy ? c - __shfl_sync(kAll, c, __ffs(heavy) - 1) : c;
        };
        const float top = warp_max(x);
        float d;
        if (!a.sigmoid) {
            float w = on && x != -INFINITY ? expf(x - top) : 0.0f;
            w = w / fmaxf(warp_sum(w), 1e-30f);
            c = less_heaviest(w);
            d = w * (c - warp_sum(w * c));
        } else if (a.renormalize) {
            const float m = fminf(top, 0.0f);
            // a NaN is not below the limit: it shows
            const float s = on && !(m < kNoSigmoid && x <= m) ? 1.0f / (expf(m) + expf(m - x)) : 0.0f;
            const float total = warp_sum(s), w = total == 0.0f ? 0.0f : s / total;
            c = less_heaviest(w);
            c -= warp_sum(w * c);
            d = w * c * (on ? sigmoid(-x) : 0.0f);
        } else {
            d = on ? c * sigmoid(x) * sigmoid(-x) : 0.0f;
        }
        if (on) atomicAdd(buf + id, d);
    }
    __syncwarp();
    T *out = static_cast<T *>(a.dlogits) + (long long)t * a.E;
    constexpr int W = 16 / (int)sizeof(T);
    float v[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) v[j] = buf[lane * VPT + j];
    if constexpr (DENSE) {
        const float c0 = first >= 0 ? buf[first] : 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            v[j] -= c0;
            dot += p[j] * v[j];
        }
        dot = warp_sum(dot);
#pragma unroll
        for (int j = 0; j < VPT; ++j) v[j] = p[j] * (v[j] - dot);
    }
    if constexpr (VPT >= W) {
        if (a.vec) {
#pragma unroll
            for (int q = 0; q < VPT / W; ++q) {
                union { uint4 u; T e[W]; } pack;
#pragma unroll
                for (int j = 0; j < W; ++j) pack.e[j] = from_f32<T>(v[q * W + j]);
                const int i = lane * VPT + q * W;
                if (i < a.E) *reinterpret_cast<uint4 *>(out + i) = pack.u;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = lane * VPT + j;
        if (i < a.E) out[i] = from_f32<T>(v[j]);
    }
}

template <typename T, int VPT>
cudaError_t route_vpt(const RouteArgs &a, bool pdl, cudaStream_t st)
{
    const dim3 grid((unsigned)((a.T + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool sums = a.bias || (a.groups > 1 && a.group_top > 1);
    if (sums) return launch_kernel(route_kernel<T, VPT, true>, grid, block, 0, pdl, 1, st, a);
    return launch_kernel(route_kernel<T, VPT, false>, grid, block, 0, pdl, 1, st, a);
}

template <typename T, int VPT>
cudaError_t backward_vpt(const RouteBackwardArgs &a, bool pdl, cudaStream_t st)
{
    const dim3 grid((unsigned)((a.T + kWarps - 1) / kWarps)), block(kWarps * 32);
    if (!a.sigmoid && !a.renormalize)
        return launch_kernel(route_backward_kernel<T, VPT, true>, grid, block, 0, pdl, 1, st, a);
    return launch_kernel(route_backward_kernel<T, VPT, false>, grid, block, 0, pdl, 1, st, a);
}

// The smallest power of two of experts per lane that holds the row.
#define BN_BY_EXPERTS(call, T, a)                     \
    ((a).E <= 32    ? call<T, 1>(a, pdl, st)          \
     : (a).E <= 64  ? call<T, 2>(a, pdl, st)          \
     : (a).E <= 128 ? call<T, 4>(a, pdl, st)          \
     : (a).E <= 256 ? call<T, 8>(a, pdl, st)          \
     : (a).E <= 512 ? call<T, 16>(a, pdl, st)         \
                    : call<T, 32>(a, pdl, st))

}  // namespace

cudaError_t launch_route(const RouteArgs &a, int dtype, bool pdl, cudaStream_t st)
{
    if (dtype == 0) return BN_BY_EXPERTS(route_vpt, __nv_bfloat16, a);
    if (dtype == 1) return BN_BY_EXPERTS(route_vpt, __half, a);
    return BN_BY_EXPERTS(route_vpt, float, a);
}

cudaError_t launch_route_backward(const RouteBackwardArgs &a, int dtype, bool pdl, cudaStream_t st)
{
    if (dtype == 0) return BN_BY_EXPERTS(backward_vpt, __nv_bfloat16, a);
    if (dtype == 1) return BN_BY_EXPERTS(backward_vpt, __half, a);
    return BN_BY_EXPERTS(backward_vpt, float, a);
}

}  // namespace bn
