// bn_swiglu.cu -- the gated activation between an expert's two layers, and its gradient.
//
// A row of x is gate and up side by side (F values each); with s = 1 / (1 + exp(-gate)):
//   y = (gate * s) * up
//   dup = dy * (gate * s),  dgate = dy * up * (s * (1 + gate * (1 - s)))
// in 32 bits, rounded once.  s and 1 - s come from z = exp(-|gate|) as 1 / (1 + z) and
// z / (1 + z), either way round, so that neither loses digits nor overflows; the
// division is the fast one (2 ulp).
//
// Memory bounds it: 3 (gradient: 5) values moved for some 20 (30) instructions.  A thread
// takes 16 bytes of each operand at a time; rows whose length or alignment does not allow that
// go value by value.  32768 rows of 2048: 74 us with 8 blocks an SM that stride (60 at the
// copy rate; 78 with a block for every 256 vectors, 80 with two vectors in flight a thread),
// the gradient 96 with a block for every 256 vectors (100 at the copy rate, but the last of its output
// stays in L2; 117 striding).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {
using namespace dev;

namespace {

template <typename T> __device__ __forceinline__ float widen(T v) { return (float)v; }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V values of T, moved together.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T>
__device__ __forceinline__ void one(float gate, float up, float dy, bool backward, T &a, T &b)
{
    const float z = expf(-fabsf(gate)), r = __fdividef(1.0f, 1.0f + z), q = z * r;
    const float s = gate >= 0.0f ? r : q, t = gate >= 0.0f ? q : r;  // t = 1 - s
    const float silu = gate * s;
    if (!backward) {
        a = narrow<T>(silu * up);
        return;
    }
    a = narrow<T>(dy * up * (s + silu * t));
    b = narrow<T>(dy * silu);
}

template <typename T, int V, bool BACKWARD>
__global__ void __launch_bounds__(256) swiglu_kernel(const __grid_constant__ SwigluArgs p)
{
    using P = Pack<T, V>;
    griddep_launch_dependents();
    griddep_wait();
    const unsigned per = (unsigned)(p.F / V);
    const long long total = (long long)p.M * per, step = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        // 32-bit division where the index fits
        const long long m = total >> 32 ? i / per : (unsigned)i / per;
        const int f = (int)(i - m * per) * V;
        const T *x = static_cast<const T *>(p.x) + m * p.ld + f;
        const P gate = *reinterpret_cast<const P *>(x), up = *reinterpret_cast<const P *>(x + p.F);
        P dy = {}, a, b;
        if (BACKWARD) dy = *reinterpret_cast<const P *>(static_cast<const T *>(p.dy) + m * p.ld_dy + f);
#pragma unroll
        for (int j = 0; j < V; ++j)
            one<T>(widen(gate.v[j]), widen(up.v[j]), BACKWARD ? widen(dy.v[j]) : 0.0f, BACKWARD, a.v[j], b.v[j]);
        if (BACKWARD) {
            T *out = static_cast<T *>(p.out) + m * 2 * p.F + f;
            *reinterpret_cast<P *>(out) = a;
            *reinterpret_cast<P *>(out + p.F) = b;
        } else {
            *reinterpret_cast<P *>(static_cast<T *>(p.out) + m * p.F + f) = a;
        }
    }
}

template <typename T, int V>
cudaError_t launch_type(const SwigluArgs &p, bool backward, int sms, bool pdl, cudaStream_t st)
{
    auto *k = backward ? swiglu_kernel<T, V, true> : swiglu_kernel<T, V, false>;
    const long long blocks = ((long long)p.M * (p.F / V) + 255) / 256, most = backward ? (1LL << 31) - 1 : 8LL * sms;
    return launch_kernel(k, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, pdl, 1, st, p);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs &p, int dtype, bool backward, int sms, bool pdl, cudaStream_t st)
{
    switch (dtype) {
    case 0: return p.vec ? launch_type<__nv_bfloat16, 8>(p, backward, sms, pdl, st) : launch_type<__nv_bfloat16, 1>(p, backward, sms, pdl, st);
    case 1: return p.vec ? launch_type<__half, 8>(p, backward, sms, pdl, st) : launch_type<__half, 1>(p, backward, sms, pdl, st);
    default: return p.vec ? launch_type<float, 4>(p, backward, sms, pdl, st) : launch_type<float, 1>(p, backward, sms, pdl, st);
    }
}

}  // namespace bn
