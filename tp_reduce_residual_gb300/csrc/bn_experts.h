// bn_experts.h -- the operators around the experts: launch arguments shared by
// the ABI (bn_experts_abi.cu) and the kernels (bn_route.cu, bn_plan.cu,
// bn_fp4.cu, bn_product.cu).  Not part of the ABI.
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

// dtype: 0 BF16, 1 FP16, 2 FP32.  fmt: 0 NVFP4, 1 MXFP4.
cudaError_t launch_route(const RouteArgs &, int dtype, bool pdl, cudaStream_t);
cudaError_t launch_route_backward(const RouteBackwardArgs &, int dtype, bool pdl, cudaStream_t);
cudaError_t launch_plan(const PlanArgs &, bool pdl, cudaStream_t);
cudaError_t launch_quantize(const QuantArgs &, int dtype, int fmt, int sms, bool pdl, cudaStream_t);
cudaError_t launch_dequantize(const QuantArgs &, int dtype, int fmt, int sms, bool pdl, cudaStream_t);
cudaError_t launch_product(const ProductArgs &, const uint8_t *a, const uint8_t *w, int fmt, int sms,
                           bool pdl, cudaStream_t);

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
