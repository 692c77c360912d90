// bn_int8.cu -- rows in 8-bit integers with a scale a row: quantisation and back.
//
// With top = max |x| of a row, scale = top / 127 rounded to FP32, and a code is the whole
// number nearest to x / scale, half way to the even one: the choice of exact arithmetic.
// y = x * (1 / scale) is off by at most 127 * 2^-22; only where it is within 10^-4 of
// half way is the remainder x - code * scale taken, which one FMA gives exactly (a
// multiple of the smaller of the two last places, below half a scale), and compared with half
// the scale.  Rows below 2^-60 are scaled by 2^100 first, exactly, so that 1 / scale is
// finite.  A row with an infinity or a NaN gets a NaN scale and codes 0; a row of
// zeros scale 0.
//
// Between 32 and 256 threads a row hold up to 128 bytes of it each in registers, so that
// it is read once; what a longer row has beyond that is read again from L2.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {
using namespace dev;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kHeld = 8;  // vectors of 16 bytes that a thread holds

template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    static __device__ __forceinline__ void widen(const uint4 &q, float *v)
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same_v<T, __half>) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = h.x, v[2 * i + 1] = h.y;
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// The bits of the largest magnitude: infinities and NaN are above every number.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint4 &q, uint32_t top)
{
    float v[Vec<T>::kN];
    Vec<T>::widen(q, v);
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    return top;
}

struct RowScale {
    float up, scale, inv, half;  // values and scale times `up`
};

__device__ __forceinline__ int code_of(float x, const RowScale &s)
{
    x *= s.up;
    const float y = x * s.inv, q = rintf(y);
    int code = (int)q;
    if (fabsf(y - q) > 0.4999f) {
        const float r = fabsf(fmaf(-q, s.scale, x));
        // the other neighbour: nearer, or as near and even
        if (r > s.half || (r == s.half && (code & 1))) code += fmaf(-q, s.scale, x) > 0.0f ? 1 : -1;
    }
    return min(max(code, -127), 127);
}

template <typename T>
__device__ __forceinline__ void store_codes(int8_t *to, const uint4 &q, const RowScale &s)
{
    float v[Vec<T>::kN];
    Vec<T>::widen(q, v);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; ++i) w[i / 4] |= ((uint32_t)code_of(v[i], s) & 0xffu) << (8 * (i & 3));
    if constexpr (Vec<T>::kN == 8)
        *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(to) = w[0];
}

// W: threads of a row.
template <typename T, int W>
__global__ void __launch_bounds__(256) quantize_int8_kernel(const __grid_constant__ Int8Args a)
{
    constexpr int kRowsPer = 256 / W, kN = Vec<T>::kN;
    __shared__ uint32_t tops[8];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, at = threadIdx.x % W;
    const int m = blockIdx.x * kRowsPer + threadIdx.x / W;
    const bool live = m < a.M;  // of a block of several rows, the last ones may be past the end
    long long src = live ? m : 0;
    if (live && a.rows) {
        src = __ldg(a.rows + m);
        if (src < 0 || src >= a.x_rows) {
            if (at == 0) atomicOr(a.err, BN_DEVERR_PERM_RANGE);
            src = 0;
        }
    }
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + src * a.ld);
    const int n = a.K / kN;
    uint4 held[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = at + i * W;
        held[i] = make_uint4(0, 0, 0, 0);
        if (j < n) held[i] = __ldg(x + j);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) top = top_bits<T>(held[i], top);
    for (int j = at + kHeld * W; j < n; j += W) top = top_bits<T>(__ldg(x + j), top);
    top = __reduce_max_sync(kAll, top);
    if constexpr (W > 32) {
        if (lane == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        constexpr int kWarps = W / 32;
        const int first = (int)(threadIdx.x / W) * kWarps;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = max(top, tops[first + i]);
    }
    if (!live) return;
    const bool bad = top >= 0x7f800000u;
    const float amax = __uint_as_float(top), scale = __fdiv_rn(amax, 127.0f);
    RowScale s;
    s.up = bad ? 0.0f : amax < 0x1p-60f ? 0x1p100f : 1.0f;
    s.scale = scale * s.up;
    s.half = 0.5f * s.scale;
    s.inv = bad || scale == 0.0f ? 0.0f : __frcp_rn(s.scale);
    if (at == 0) a.scales[m] = bad ? __uint_as_float(0x7fc00000u) : scale;
    int8_t *to = a.data + (long long)m * a.K;
    if (bad || scale == 0.0f) {
        for (int j = at; j < n; j += W) {
            if constexpr (kN == 8) reinterpret_cast<uint2 *>(to)[j] = make_uint2(0, 0);
            else reinterpret_cast<uint32_t *>(to)[j] = 0;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int j = at + i * W;
        if (j < n) store_codes<T>(to + (long long)j * kN, held[i], s);
    }
    for (int j = at + kHeld * W; j < n; j += W) store_codes<T>(to + (long long)j * kN, __ldg(x + j), s);
}

// 16 codes a thread.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_int8_kernel(const __grid_constant__ Int8Args a)
{
    griddep_launch_dependents();
    griddep_wait();
    const unsigned per = (unsigned)a.K / 16;
    const long long total = (long long)a.M * per, step = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
        const long long m = total >> 32 ? i / per : (unsigned)i / per;
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a.data) + i);
        const float scale = __ldg(a.scales + m);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        alignas(16) T v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = (T)((float)(int8_t)(w[j / 4] >> (8 * (j & 3))) * scale);
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + i * 16);
#pragma unroll
        for (int j = 0; j < (int)sizeof(T); ++j) out[j] = reinterpret_cast<const uint4 *>(v)[j];
    }
}

template <typename T>
cudaError_t launch_quantize_type(const Int8Args &a, bool pdl, cudaStream_t st)
{
    const int n = a.K / Vec<T>::kN;
    const auto go = [&](auto *k, int w) {
        return launch_kernel(k, dim3((unsigned)((a.M + 256 / w - 1) / (256 / w))), dim3(256), 0, pdl, 1, st, a);
    };
    if (n <= 32 * kHeld) return go(quantize_int8_kernel<T, 32>, 32);
    if (n <= 128 * kHeld) return go(quantize_int8_kernel<T, 128>, 128);
    return go(quantize_int8_kernel<T, 256>, 256);
}

}  // namespace

cudaError_t launch_quantize_int8(const Int8Args &a, int dtype, bool pdl, cudaStream_t st)
{
    return dtype == 0 ? launch_quantize_type<__nv_bfloat16>(a, pdl, st)
         : dtype == 1 ? launch_quantize_type<__half>(a, pdl, st) : launch_quantize_type<float>(a, pdl, st);
}

cudaError_t launch_dequantize_int8(const Int8Args &a, int dtype, int sms, bool pdl, cudaStream_t st)
{
    const long long blocks = ((long long)a.M * (a.K / 16) + 255) / 256, most = 16LL * sms;
    auto *k = dtype == 0 ? dequantize_int8_kernel<__nv_bfloat16> : dtype == 1 ? dequantize_int8_kernel<__half> : dequantize_int8_kernel<float>;
    return launch_kernel(k, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, pdl, 1, st, a);
}

}  // namespace bn
