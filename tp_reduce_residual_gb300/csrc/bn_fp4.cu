// bn_fp4.cu -- microscaled 4-bit floating point: quantisation and back.
//
// A value is code * block scale * tensor scale.  The codes are 4-bit floats
// (sign, 2 exponent bits, 1 mantissa bit: 0 0.5 1 1.5 2 3 4 6).
//   NVFP4: blocks of 16 along a row; the scale is the 8-bit float with 4
//     exponent bits (e4m3) next to max|x| / 6, at most 448.
//   MXFP4: blocks of 32; the scale is 2^(floor(log2 max|x|) - 2).
// Codes are x / scale rounded to the nearest, half way to the even code, at
// most 6.  The tensor scale is a power of two, so dividing by it is exact, and
// every choice below is the one exact arithmetic makes for BF16 and FP16
// values: a half-way point times a scale has at most 7 significant bits and x
// at most 11, so a quotient that is not half way is at least 2^-12 of itself
// away from it, far beyond a rounding of 2^-24, and a quotient that is half way
// is exact because it is corrected once with its remainder.
// A block with an infinity or a NaN gets a NaN scale: its values are NaN.
//
// Codes are stored two a byte, the even element in the low half, rows of K / 2
// bytes.  Scales are stored as the tensor core reads them: in tiles of 128 rows
// by 4 scales (512 bytes, row r of the tile at (r % 32) * 16 + (r / 32) * 4),
// tiles of the same rows in the order of K, and the row tiles of group g from
// tile (offsets[g] >> 7) + g on, which leaves every group its own tiles without
// a sum over the groups.  Scales past the end of a row are 0.
//
// One warp per row (or per share of a row): a lane takes 16 values, the four
// lanes of a scale tile row join their scale bytes into one 4-byte store.  DRAM
// bandwidth bounds it at many rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/beamnorm.h"
#include "bn_device.cuh"
#include "bn_experts.h"

namespace bn {
using namespace dev;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRowWarps = 4;

template <typename T> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    static __device__ __forceinline__ float2 widen(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static constexpr uint32_t kInf = 0x7f80u;
};
template <> struct Half2<__half> {
    static __device__ __forceinline__ float2 widen(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static constexpr uint32_t kInf = 0x7c00u;
};

// The row's place among the scale tiles.  The group is the number of group ends
// at or below m (a warp-wide count, in bounds whatever the offsets hold).
struct Place {
    int tile, r;
};
__device__ __forceinline__ Place place_of(const QuantArgs &a, int m, int lane)
{
    int g, start;
    if (a.offsets) {
        int n = 0;
        for (int i = lane; i < a.groups; i += 32) n += __ldg(a.offsets + 1 + i) <= m ? 1 : 0;
        g = __reduce_add_sync(kAll, n);
        start = min(max(__ldg(a.offsets + g), 0), m);
        const int r = m - start;
        return {(start >> 7) + g + (r >> 7), r & 127};
    }
    g = m / a.per;
    const int r = m - g * a.per;
    return {g * a.tiles_per + (r >> 7), r & 127};
}

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tcvt.u32.u8 %0, q;\n\t}"
        : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// The e4m3 byte next to v >= 0, at most 448.
__device__ __forceinline__ uint32_t e4m3(float v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(v), "f"(0.0f));
    return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}
// 2^(code - 127); code 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code)
{
    return __uint_as_float(code == 255u ? 0x7fc00000u : code ? code << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    return __vmaxu2(a, b & 0x7fff7fffu);
}

template <typename T, bool MX>
__global__ void __launch_bounds__(kRowWarps * 32) quantize_kernel(QuantArgs a, int chunks, int share)
{
    const int lane = threadIdx.x & 31;
    const int m = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    griddep_launch_dependents();
    griddep_wait();
    if (m >= a.M) return;
    long long src = m;
    if (a.rows) {
        src = __ldg(a.rows + m);
        if (src < 0 || src >= a.x_rows) {
            if (lane == 0) atomicOr(a.err, BN_DEVERR_PERM_RANGE);
            src = 0;
        }
    }
    const Place p = place_of(a, m, lane);
    const T *x = static_cast<const T *>(a.x) + src * a.ld;
    uint8_t *data = a.data + (long long)m * (a.K / 2);
    // scales of this row: 4 bytes of every 512-byte tile
    uint8_t *scales = a.scales + ((long long)p.tile * chunks) * 512 + (p.r & 31) * 16 + (p.r >> 5) * 4;
    constexpr int kChunk = MX ? 128 : 64;  // values of a row in one scale tile
    const int end = chunks * kChunk;       // the padded row: its last scales are written as 0
    const int k1 = min(end, (int)(blockIdx.y + 1) * share);
    for (int k0 = blockIdx.y * share; k0 < k1; k0 += 512) {
        const int k = k0 + lane * 16;
        uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;
        if (k < a.K) q0 = __ldg(reinterpret_cast<const uint4 *>(x + k));
        if (k < a.K) q1 = __ldg(reinterpret_cast<const uint4 *>(x + k + 8));
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t top2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top2 = max_abs2(top2, w[i]);
        uint32_t top = max(top2 & 0xffffu, top2 >> 16);  // bits of the largest magnitude
        if (MX) top = max(top, __shfl_xor_sync(kAll, top, 1));
        const bool bad = top >= Half2<T>::kInf;
        const float amax = Half2<T>::widen(top).x * a.inv_tensor_scale;
        uint32_t code;
        float mul, scale = 1.0f;  // x * mul / scale is what is rounded
        if (MX) {
            const int e = (int)(__float_as_uint(amax) >> 23);  // exponent field; 0: nothing to scale
            code = bad ? 255u : (uint32_t)max(e - 2, 0);
            // 2^(127 - code), a subnormal for code 254
            mul = __uint_as_float(code >= 254u ? 0x00400000u : (254u - code) << 23);
        } else {
            code = bad ? 0x7fu : e4m3(__fdiv_rn(amax, 6.0f));
            scale = e4m3_value(code);
            mul = bad || code == 0 ? 0.0f : __frcp_rn(scale);
        }
        if (bad) mul = 0.0f;
        uint32_t packed[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 v = Half2<T>::widen(w[i]);
            v.x *= a.inv_tensor_scale;
            v.y *= a.inv_tensor_scale;
            float2 y = make_float2(v.x * mul, v.y * mul);
            if (!MX) {  // the remainder makes an exact quotient exact
                y.x = __fmaf_rn(__fmaf_rn(-y.x, scale, v.x), mul, y.x);
                y.y = __fmaf_rn(__fmaf_rn(-y.y, scale, v.y), mul, y.y);
            }
            packed[i >> 2] |= e2m1x2(y.x, y.y) << (8 * (i & 3));
        }
        if (bad) packed[0] = packed[1] = 0;
        if (k < a.K) *reinterpret_cast<uint2 *>(data + k / 2) = make_uint2(packed[0], packed[1]);
        if (k >= a.K) code = 0;
        // four scales of one tile row: of lanes 0..3 of four (NVFP4) or of every second of eight (MXFP4)
        uint32_t word;
        if (MX) {
            word = code | (__shfl_down_sync(kAll, code, 2) << 8);
            word |= __shfl_down_sync(kAll, word, 4) << 16;
        } else {
            word = code | (__shfl_down_sync(kAll, code, 1) << 8);
            word |= __shfl_down_sync(kAll, word, 2) << 16;
        }
        if ((lane & (MX ? 7 : 3)) == 0 && k < end)
            *reinterpret_cast<uint32_t *>(scales + (long long)(k / kChunk) * 512) = word;
    }
}

template <typename T> __device__ __forceinline__ void store16(T *out, const float *v);
template <> __device__ __forceinline__ void store16(float *out, const float *v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4 *>(out)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <> __device__ __forceinline__ void store16(__nv_bfloat16 *out, const float *v)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint4 *>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <> __device__ __forceinline__ void store16(__half *out, const float *v)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    reinterpret_cast<uint4 *>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T, bool MX>
__global__ void __launch_bounds__(kRowWarps * 32) dequantize_kernel(QuantArgs a, int chunks, int share)
{
    const int lane = threadIdx.x & 31;
    const int m = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    griddep_launch_dependents();
    griddep_wait();
    if (m >= a.M) return;
    const Place p = place_of(a, m, lane);
    const uint8_t *data = a.data + (long long)m * (a.K / 2);
    const uint8_t *scales = a.scales + ((long long)p.tile * chunks) * 512 + (p.r & 31) * 16 + (p.r >> 5) * 4;
    T *out = static_cast<T *>(a.out) + (long long)m * a.K;
    constexpr int kChunk = MX ? 128 : 64;
    const int k1 = min(a.K, (int)(blockIdx.y + 1) * share);
    for (int k0 = blockIdx.y * share; k0 < k1; k0 += 512) {
        const int k = k0 + lane * 16;
        if (k >= k1) break;
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(data + k / 2));
        const uint32_t b = scales[(long long)(k / kChunk) * 512 + k % kChunk / (MX ? 32 : 16)];
        const float s = (MX ? e8m0_value(b) : e4m3_value(b)) * a.tensor_scale;
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = ((i < 4 ? q.x : q.y) >> (8 * (i & 3))) & 0xffu;
            uint32_t h;
            asm("{\n\t.reg .b8 q;\n\tcvt.u8.u32 q, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;\n\t}" : "=r"(h) : "r"(byte));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
        store16<T>(out + k, v);
    }
}

// Values per block of a row: whole rows when there are warps enough for the
// device, else shares of 512 values and more.
void split_rows(const QuantArgs &a, int sms, dim3 *grid, int *share)
{
    const int blocks = (a.M + kRowWarps - 1) / kRowWarps;
    const int steps = (a.K + 511) / 512;
    int parts = 1;
    while (parts < steps && (long long)blocks * parts * kRowWarps < (long long)sms * 32) parts *= 2;
    parts = parts < steps ? parts : steps;
    const int each = (steps + parts - 1) / parts;
    *share = each * 512;
    *grid = dim3((unsigned)blocks, (unsigned)((steps + each - 1) / each));
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs &a, int dtype, int fmt, int sms, bool pdl, cudaStream_t st)
{
    dim3 grid;
    int share;
    split_rows(a, sms, &grid, &share);
    const int per = fmt ? 128 : 64, chunks = (a.K + per - 1) / per;
    auto *k = dtype == 0 ? (fmt ? quantize_kernel<__nv_bfloat16, true> : quantize_kernel<__nv_bfloat16, false>)
                         : (fmt ? quantize_kernel<__half, true> : quantize_kernel<__half, false>);
    return launch_kernel(k, grid, dim3(kRowWarps * 32), 0, pdl, 1, st, a, chunks, share);
}

cudaError_t launch_dequantize(const QuantArgs &a, int dtype, int fmt, int sms, bool pdl, cudaStream_t st)
{
    dim3 grid;
    int share;
    split_rows(a, sms, &grid, &share);
    const int per = fmt ? 128 : 64, chunks = (a.K + per - 1) / per;
    auto *k = dtype == 0   ? (fmt ? dequantize_kernel<__nv_bfloat16, true> : dequantize_kernel<__nv_bfloat16, false>)
              : dtype == 1 ? (fmt ? dequantize_kernel<__half, true> : dequantize_kernel<__half, false>)
                           : (fmt ? dequantize_kernel<float, true> : dequantize_kernel<float, false>);
    return launch_kernel(k, grid, dim3(kRowWarps * 32), 0, pdl, 1, st, a, chunks, share);
}

}  // namespace bn
