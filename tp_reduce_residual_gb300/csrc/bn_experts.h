// bn_experts.h -- the operators around the experts: launch arguments shared by
// the ABI (bn_experts_abi.cu) and the kernels (bn_route.cu, bn_plan.cu,
// bn_fp4.cu, bn_product.cu, bn_linear.cu, bn_swiglu.cu, bn_int8.cu, bn_product8.cu).  Not part of the ABI.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace bn {

constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 32;      // routing groups: one lane each

struct RouteArgs {
    const void *logits;
    long long ld;          // elements between rows
    int T, E, k;
    const float *bias;     // [E] or null
    int sigmoid;           // score: 0 softmax, 1 sigmoid
    int groups, top_groups, group_top;
    int renormalize;
    float scale;
    int R;
    int32_t *ids;          // [T, k]
    float *w;              // [R, T, k]
    int vec;               // rows are 16-byte aligned and E is a multiple of a vector
    int bias_vec;          // so is the bias
};

struct RouteBackwardArgs {
    const void *logits;
    long long ld;
    int T, E, k;
    const int32_t *ids;    // [T, k]
    const float *dw;       // [R, T, k]
    int R;
    int sigmoid, renormalize;
    float scale;
    void *dlogits;         // [T, E]
    unsigned *err;
    int vec;               // logits rows as RouteArgs::vec, and dlogits rows too
};

struct PlanArgs {
    const int32_t *ids;    // [T, k]
    int slots;             // T * k
    int k, E, R;
    int32_t *perm;         // [R, T, k]
    int32_t *offsets;      // [E + 1]
    int32_t *rows;         // [T * k]
    unsigned *err;
};

struct QuantArgs {
    const void *x;         // [x_rows, K], ld elements between rows (quantise) -- or null
    long long ld;
    long long x_rows;
    const int32_t *rows;   // [M] or null
    int M, K;
    const int32_t *offsets;  // [groups + 1] or null: groups of `per` rows
    int groups, per, tiles_per;
    float tensor_scale, inv_tensor_scale;
    uint8_t *data;         // [M, K / 2]
    uint8_t *scales;       // [tiles, chunks, 512]
    uint8_t *work;         // or null: the rows of x quantised once (codes, then scale bytes side by side)
    void *out;             // [M, K] (dequantise)
    unsigned *err;
};

struct ProductArgs {
    int M, E, N, K;
    const int32_t *offsets;   // [E + 1] or null (E = 1, all rows)
    const uint8_t *a_scales, *w_scales;
    long long a_tiles;        // row tiles of a_scales
    int chunks;               // scale chunks of 512 bytes per row tile
    float alpha;
    uint16_t *out;            // [M, N] BF16
    unsigned *err;
};

// One product of an expert's linear layer.  Forward: out [M, F] = x [M, D] of rows of a
// group times w [E, F, D]; input gradient: out [M, F] = dy [M, D] times w [E, D, F];
// weight gradient: out [E, F, K] = dy [M, F] transposed times x [M, K], group by group.
struct LinearArgs {
    int M, E, F, D, K;
    const int32_t *offsets;   // [E + 1] or null (E = 1, all rows)
    const int32_t *rows;      // [M] or null: the row of x at each place
    int x_rows;
    void *out;
    int dtype;                // of the operands: 0 BF16, 1 FP16
    int out_fp32, accumulate; // weight gradient
    int split;                // CTAs that share a tile's sum
    unsigned *err;
};
enum LinearMode { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

// A sum of d values is taken in stages of kSumStage, and those in runs of 2^log stages, of
// which a sum of no values has one.  Runs are counted from stages: d + 64 * 2^log leaves 31 bits
// at the longest sums, the rows of a call (2^31 - 1024).
constexpr int kSumStage = 64;
__host__ __device__ constexpr int sum_stages(int d) { return (d + kSumStage - 1) / kSumStage; }
__host__ __device__ constexpr int sum_runs(int d, int log) { return d > 0 ? (sum_stages(d) + (1 << log) - 1) >> log : 1; }

struct SwigluArgs {
    const void *x;         // [M, 2 F], ld elements between rows: gate and up
    const void *dy;        // [M, F], ld_dy elements between rows (gradient) -- or null
    void *out;             // [M, F], or the gradient [M, 2 F]
    long long ld, ld_dy;
    int M, F;
    int vec;               // 16-byte vectors fit every row of every operand
};

struct Int8Args {
    const void *x;         // [x_rows, K], ld elements between rows (quantise)
    long long ld;
    long long x_rows;
    const int32_t *rows;   // [M] or null
    int M, K;
    int8_t *data;          // [M, K]
    float *scales;         // [M]
    void *out;             // [M, K] (dequantise)
    unsigned *err;
};

struct Product8Args {
    int M, E, N, K;
    const int32_t *offsets;   // [E + 1] or null (E = 1, all rows)
    const int8_t *a;          // [M, K]
    const float *a_scales;    // [M]
    const float *w_scales;    // [E, N]
    float alpha;
    uint16_t *out;            // [M, N] BF16
    int split;                // CTAs that share a tile's sum
    unsigned *err;
};

// dtype: 0 BF16, 1 FP16, 2 FP32.  fmt: 0 NVFP4, 1 MXFP4.
cudaError_t launch_route(const RouteArgs &, int dtype, bool pdl, cudaStream_t);
cudaError_t launch_route_backward(const RouteBackwardArgs &, int dtype, bool pdl, cudaStream_t);
cudaError_t launch_plan(const PlanArgs &, bool pdl, cudaStream_t);
cudaError_t launch_quantize(const QuantArgs &, int dtype, int fmt, int sms, bool pdl, cudaStream_t);
cudaError_t launch_dequantize(const QuantArgs &, int dtype, int fmt, int sms, bool pdl, cudaStream_t);
cudaError_t launch_product(const ProductArgs &, const uint8_t *a, const uint8_t *w, int fmt, int sms,
                           bool pdl, cudaStream_t);

// x: the rows operand (x, or dy), ld elements between rows; w: the weights, or for the
// weight gradient dy, w_ld elements between rows.
cudaError_t launch_linear(const LinearArgs &, LinearMode mode, const void *x, long long ld, const void *w, long long w_ld,
                          int sms, bool pdl, cudaStream_t);

cudaError_t launch_swiglu(const SwigluArgs &, int dtype, bool backward, int sms, bool pdl, cudaStream_t);
cudaError_t launch_quantize_int8(const Int8Args &, int dtype, bool pdl, cudaStream_t);
cudaError_t launch_dequantize_int8(const Int8Args &, int dtype, bool pdl, cudaStream_t);
// Whether pairs of CTAs serve the product; `split`: the CTAs that share a tile's sum, if not.
bool product8_pairs(const Product8Args &, int sms, int *split);
// workspace: 2 M K bytes, for the rows widened to FP16 where pairs serve, or null: no pairs.
cudaError_t launch_product8(Product8Args, const int8_t *w, void *workspace, int sms, bool pdl, cudaStream_t);
// out [M, K] dense: row rows[m] of x at place m (16-bit values); likewise its scale, if scales are given.
// With the groups' offsets [E + 1], indexes outside x are errors at places of groups alone.
cudaError_t launch_place_rows(const void *x, long long ld, int x_rows, const int32_t *rows, int M, const int32_t *offsets, int E, int K,
                              void *out, const float *scales, float *out_scales, unsigned *err, int sms, bool pdl, cudaStream_t st);

// A kernel's attributes, set once per device: dynamic shared memory of up to
// `bytes`, and clusters of more than 8 CTAs if `wide`.
class KernelSetup {
public:
    template <typename... P>
    cudaError_t operator()(void (*kernel)(P...), int bytes, bool wide = false)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && wide) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<unsigned long long> done_{0};
};

// One launch, with or without programmatic dependent launch.
template <typename... P, typename... A>
inline cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, bool pdl,
                                 int cluster, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (pdl) {
        at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = (unsigned)cluster;
        at[n].val.clusterDim.y = 1;
        at[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = (unsigned)n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace bn
