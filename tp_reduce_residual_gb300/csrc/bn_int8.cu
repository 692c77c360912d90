// bn_int8.cu -- rows in 8-bit integers with a scale a row: quantisation and back.
//
// With top = max |x| of a row, scale = top / 127 rounded to FP32, and a code is the whole
// number nearest to x / scale, half way to the even one: the choice of exact arithmetic.
// x * (1 / scale) is off by at most 127 * 2^-22, so the whole number next to it (one FMA with
// 1.5 * 2^23) is the code or, near half way, its neighbour.  The remainder x - code * scale is
// exact in one FMA (a multiple of the smaller of the two last places, about half a scale at
// most); where it reaches half the scale, eight codes are decided again, one by one.  Rows below
// 2^-60 are scaled by 2^100 first, exactly, so that 1 / scale is finite.  A row with an
// infinity or a NaN gets a NaN scale and codes 0; a row of zeros scale 0.
//
// Between 32 and 256 threads a row hold up to 128 bytes of it each in registers, so that
// it is read once; what a longer row has beyond that is read again from L2.  Memory bounds
// rows in their places: 32768 of 5120 in 88 us (75 at the copy rate), 32768 of 2048 in 37
// (30).  Rows repeated from 4096 come from L2, in 80 us: about 7 instructions a value and
// the wait for the row's largest; quantised once into a workspace and copied 42.  Between 64 and 128 bytes a thread: with 8 vectors held for
// rows of 5 a thread 92 us, with a warp a row of 20 a thread 117.
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

// The larger magnitudes of two words of values, NaN the largest; in 16 bits the signs are of no use.
template <typename T> __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t larger<float>(uint32_t a, uint32_t b) { return max(a & 0x7fffffffu, b & 0x7fffffffu); }
template <> __device__ __forceinline__ uint32_t larger<__nv_bfloat16>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t larger<__half>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t larger(const uint4 &q, uint32_t top)
{
    return larger<T>(larger<T>(q.x, q.y), larger<T>(larger<T>(q.z, q.w), top));
}
// The FP32 bits of the largest magnitude of such a word: infinities and NaN are above every number.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(uint32_t w)
{
    if constexpr (sizeof(T) == 4) {
        return w & 0x7fffffffu;
    } else {
        const uint32_t h = max(w & 0x7fffu, (w >> 16) & 0x7fffu);
        if constexpr (std::is_same_v<T, __half>) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
        return h << 16;
    }
}

struct RowScale {
    float up, scale, inv, half;  // values are taken times `up`; the rest is for those
};

// The code of x (times up already), decided exactly.
__device__ __forceinline__ uint32_t code_of(float x, const RowScale &s)
{
    const float y = x * s.inv, q = rintf(y), d = fmaf(-q, s.scale, x), r = fabsf(d);
    int code = (int)q;
    // the other neighbour: nearer, or as near and even
    if (r > s.half || (r == s.half && (code & 1))) code += d > 0.0f ? 1 : -1;
    return (uint32_t)min(max(code, -127), 127) & 0xffu;
}

// SMALL: rows of small values, which are scaled up first and may leave the range of codes.
template <typename T, bool SMALL>
__device__ __forceinline__ void store_codes(int8_t *to, const uint4 &q, const RowScale &s)
{
    constexpr int kN = Vec<T>::kN;
    float v[kN];
    Vec<T>::widen(q, v);
    uint32_t w[2] = {0, 0};
    bool exact = !SMALL;
    if (!SMALL) {
        uint32_t y[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const float near = fmaf(v[i], s.inv, 12582912.0f);  // the code in the lowest bits
            exact &= fabsf(fmaf(-(near - 12582912.0f), s.scale, v[i])) < s.half;
            y[i] = __float_as_uint(near);
        }
#pragma unroll
        for (int i = 0; i < kN; i += 4)
            w[i / 4] = __byte_perm(__byte_perm(y[i], y[i + 1], 0x0040), __byte_perm(y[i + 2], y[i + 3], 0x0040), 0x5410);
    }
    if (!exact) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i / 4] |= code_of(SMALL ? v[i] * s.up : v[i], s) << (8 * (i & 3));
    }
    if constexpr (kN == 8)
        *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint32_t *>(to) = w[0];
}

// W: threads of a row, each of which holds H vectors of 16 bytes.
template <typename T, int W, int H>
__global__ void __launch_bounds__(256, H <= 5 ? 5 : 4) quantize_int8_kernel(const __grid_constant__ Int8Args a)
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
    uint4 held[H];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const int j = at + i * W;
        held[i] = make_uint4(0, 0, 0, 0);
        if (j < n) held[i] = __ldg(x + j);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) top = larger<T>(held[i], top);
    for (int j = at + H * W; j < n; j += W) top = larger<T>(__ldg(x + j), top);
    top = __reduce_max_sync(kAll, top_bits<T>(top));
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
    const auto store = [&](auto small) {
        constexpr bool SMALL = decltype(small)::value;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int j = at + i * W;
            if (j < n) store_codes<T, SMALL>(to + (long long)j * kN, held[i], s);
        }
        for (int j = at + H * W; j < n; j += W) store_codes<T, SMALL>(to + (long long)j * kN, __ldg(x + j), s);
    };
    if (s.up != 1.0f) store(std::true_type{});
    else store(std::false_type{});
}

// A thread's codes are those of 16 bytes of values, so that every store is whole; W threads of
// a row.  32768 rows of 5120 to BF16 77 us (75 at the copy rate; 16 codes a thread, whose two
// stores are 32 bytes apart, 100).
template <typename T, int W>
__global__ void __launch_bounds__(256) dequantize_int8_kernel(const __grid_constant__ Int8Args a)
{
    constexpr int kN = Vec<T>::kN;
    using Codes = std::conditional_t<kN == 8, uint2, uint32_t>;
    griddep_launch_dependents();
    griddep_wait();
    const int m = blockIdx.x * (256 / W) + threadIdx.x / W;
    if (m >= a.M) return;
    const float scale = __ldg(a.scales + m);
    const Codes *from = reinterpret_cast<const Codes *>(a.data + (long long)m * a.K);
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + (long long)m * a.K);
    const int n = a.K / kN;
    constexpr int kAhead = 4;
    for (int j0 = threadIdx.x % W; j0 < n; j0 += kAhead * W) {
        Codes c[kAhead] = {};
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (j0 + u * W < n) c[u] = __ldg(from + j0 + u * W);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            uint32_t w[2];
            if constexpr (kN == 8) w[0] = c[u].x, w[1] = c[u].y;
            else w[0] = c[u];
            alignas(16) T v[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = (T)((float)(int8_t)(w[i / 4] >> (8 * (i & 3))) * scale);
            if (j0 + u * W < n) to[j0 + u * W] = *reinterpret_cast<const uint4 *>(v);
        }
    }
}

template <typename T>
cudaError_t launch_type(const Int8Args &a, bool back, bool pdl, cudaStream_t st)
{
    const int n = a.K / Vec<T>::kN;
    const auto go = [&](auto *k, int w) {
        return launch_kernel(k, dim3((unsigned)((a.M + 256 / w - 1) / (256 / w))), dim3(256), 0, pdl, 1, st, a);
    };
    if (back) return n <= 1024 ? go(dequantize_int8_kernel<T, 32>, 32) : go(dequantize_int8_kernel<T, 256>, 256);
    // a warp a row where it can hold one: no warp waits for another
    if (n <= 128) return go(quantize_int8_kernel<T, 32, 4>, 32);
    if (n <= 256) return go(quantize_int8_kernel<T, 32, 8>, 32);
    if (n <= 512) return go(quantize_int8_kernel<T, 128, 4>, 128);
    if (n <= 640) return go(quantize_int8_kernel<T, 128, 5>, 128);
    if (n <= 1024) return go(quantize_int8_kernel<T, 128, 8>, 128);
    return go(quantize_int8_kernel<T, 256, 8>, 256);
}

cudaError_t launch_any(const Int8Args &a, int dtype, bool back, bool pdl, cudaStream_t st)
{
    return dtype == 0 ? launch_type<__nv_bfloat16>(a, back, pdl, st)
         : dtype == 1 ? launch_type<__half>(a, back, pdl, st) : launch_type<float>(a, back, pdl, st);
}

}  // namespace

cudaError_t launch_quantize_int8(const Int8Args &a, int dtype, bool pdl, cudaStream_t st) { return launch_any(a, dtype, false, pdl, st); }
cudaError_t launch_dequantize_int8(const Int8Args &a, int dtype, bool pdl, cudaStream_t st) { return launch_any(a, dtype, true, pdl, st); }

}  // namespace bn
