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
// lanes of a scale tile row join their scale bytes into one 4-byte store.  Memory
// bounds rows in their places (32768 rows of 5120, MXFP4: 63 us, 6.7 TB/s) and the
// way back (67).  Where rows are repeated (a token's for each of its experts) they
// come from L2, and about 7 instructions a value bound it, so enough of them are
// quantised once into a workspace and copied from there: 32768 places of 4096 such
// rows take 11 us and 18, where quantising each place takes 39.
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
// at or below m (a warp-wide count, in bounds whatever the offsets hold).  A row
// before its group's start (one before the first offset) is in no group and has none.
struct Place {
    int tile, r;
    bool in;
};
__device__ __forceinline__ Place place_of(const QuantArgs &a, int m, int lane)
{
    int g, start;
    if (a.offsets) {
        int n = 0;
        for (int i = lane; i < a.groups; i += 32) n += __ldg(a.offsets + 1 + i) <= m ? 1 : 0;
        g = __reduce_add_sync(kAll, n);
        start = max(__ldg(a.offsets + g), 0);
        if (start > m) return {0, 0, false};
        const int r = m - start;
        return {(start >> 7) + g + (r >> 7), r & 127, true};
    }
    g = m / a.per;
    const int r = m - g * a.per;
    return {g * a.tiles_per + (r >> 7), r & 127, true};
}

// Eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const f2 *y)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(y[i], v[2 * i], v[2 * i + 1]);
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b16 e, f;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b16 e, {a, b};\n\tmov.b16 f, {c, d};\n\tmov.b32 %0, {e, f};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
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

// The larger magnitudes of two pairs (a NaN where there is one); the signs are of no use.
template <typename T> __device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t max_abs2<__nv_bfloat16>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <> __device__ __forceinline__ uint32_t max_abs2<__half>(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The block of 16 (half a block of 32) values in w: its codes and its scale byte.
template <typename T, bool MX>
__device__ __forceinline__ uint32_t quantize16(const uint32_t *w, float inv_tensor_scale, uint2 &codes)
{
    uint32_t top2 = max_abs2<T>(w[0], w[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) top2 = max_abs2<T>(top2, w[i]);
    uint32_t top = max(top2 & 0x7fffu, (top2 >> 16) & 0x7fffu);  // bits of the largest magnitude
    if (MX) top = max(top, __shfl_xor_sync(kAll, top, 1));
    const bool bad = top >= Half2<T>::kInf;
    const float amax = Half2<T>::widen(top).x * inv_tensor_scale;
    uint32_t code;
    float mul, scale = 1.0f;  // x * mul / scale is what is rounded
    if (MX) {
        const int e = (int)(__float_as_uint(amax) >> 23);  // exponent field; 0: nothing to scale
        code = bad ? 255u : (uint32_t)max(e - 2, 0);
        // 2^(127 - code), a subnormal for code 254
        mul = bad ? 0.0f : __uint_as_float(code >= 254u ? 0x00400000u : (254u - code) << 23);
    } else {
        code = bad ? 0x7fu : e4m3(__fdiv_rn(amax, 6.0f));
        scale = e4m3_value(code);
        mul = bad || code == 0 ? 0.0f : __frcp_rn(scale);
    }
    const f2 inv2 = f2_make(inv_tensor_scale, inv_tensor_scale), mul2v = f2_make(mul, mul), neg = f2_make(-scale, -scale);
    f2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 h = Half2<T>::widen(w[i]);
        f2 v = f2_make(h.x, h.y);
        if (inv_tensor_scale != 1.0f) v = mul2(v, inv2);
        y[i] = mul2(v, mul2v);
        if (!MX) y[i] = fma2(fma2(y[i], neg, v), mul2v, y[i]);  // the remainder makes an exact quotient exact
    }
    codes = bad ? make_uint2(0, 0) : make_uint2(e2m1x8(y), e2m1x8(y + 4));
    return code;
}

// WORK: into a workspace, whose rows have their scale bytes side by side.  The kernel
// that places them is then launched at the end: launched at the start, its first blocks,
// which write the scale tiles and last longest, were packed into the SMs that this one
// left room on (24000 places of 6000 rows of 4096 values 32 us, then 55).
template <typename T, bool MX, bool WORK>
__global__ void __launch_bounds__(kRowWarps * 32) quantize_kernel(const __grid_constant__ QuantArgs a, int chunks, int share)
{
    const int lane = threadIdx.x & 31;
    const int m = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (!WORK) griddep_launch_dependents();
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
    const Place p = WORK ? Place{0, 0, true} : place_of(a, m, lane);
    const T *x = static_cast<const T *>(a.x) + src * a.ld;
    uint8_t *data = a.data + (long long)m * (a.K / 2);
    // scales of this row: 4 bytes of every 512-byte tile
    uint8_t *scales = a.scales + (WORK ? (long long)m * chunks * 4
                                       : (long long)p.tile * chunks * 512 + (p.r & 31) * 16 + (p.r >> 5) * 4);
    constexpr unsigned kChunk = MX ? 128 : 64;  // values of a row in one scale tile
    constexpr unsigned kAhead = 2;         // steps of 512 values whose loads are in flight together
    const unsigned end = (unsigned)chunks * kChunk;  // the padded row: its last scales are written as 0
    const unsigned K = (unsigned)a.K, k1 = min(end, (blockIdx.y + 1) * (unsigned)share), inside = min(K, k1);
    unsigned k = blockIdx.y * (unsigned)share + lane * 16u;
    // `kAhead` steps from k on; FULL: all their values are inside the row
    const auto steps = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        uint32_t w[kAhead][8];
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u) {
            uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;
            if (FULL || k + 512 * u < inside) {
                q0 = __ldg(reinterpret_cast<const uint4 *>(x + k + 512 * u));
                q1 = __ldg(reinterpret_cast<const uint4 *>(x + k + 512 * u + 8));
            }
            w[u][0] = q0.x, w[u][1] = q0.y, w[u][2] = q0.z, w[u][3] = q0.w;
            w[u][4] = q1.x, w[u][5] = q1.y, w[u][6] = q1.z, w[u][7] = q1.w;
        }
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u) {
            const unsigned at = k + 512 * u;
            uint2 codes;
            uint32_t code = quantize16<T, MX>(w[u], a.inv_tensor_scale, codes);
            if (FULL || at < inside) *reinterpret_cast<uint2 *>(data + at / 2) = codes;
            if (!FULL && at >= K) code = 0;
            // four scales of one tile row: of lanes 0..3 of four (NVFP4) or of every second of eight (MXFP4)
            uint32_t word = code | (__shfl_down_sync(kAll, code, MX ? 2 : 1) << 8);
            word |= __shfl_down_sync(kAll, word, MX ? 4 : 2) << 16;
            if ((lane & (MX ? 7 : 3)) == 0 && p.in && (FULL || at < k1))
                *reinterpret_cast<uint32_t *>(scales + (size_t)(at / kChunk) * (WORK ? 4 : 512)) = word;
        }
        k += 512 * kAhead;
    };
    while (k - lane * 16u + 512 * kAhead <= inside) steps(std::true_type{});
    while (k - lane * 16u < k1) steps(std::false_type{});
    if (WORK) griddep_launch_dependents();
}

// Quantised rows from the workspace to their places.  The first `tiles` blocks
// write one scale tile row each, 16 bytes (four rows' scales) a lane: written row
// by row, 4 bytes in each 512, the scales took 8 us of 34 at 32768 rows of 5120.
// The others copy the codes, a row a warp.
__global__ void __launch_bounds__(kRowWarps * 32)
place_rows_kernel(const __grid_constant__ QuantArgs a, const uint8_t *work, const uint32_t *work_scales, unsigned chunks,
                  int tiles)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_launch_dependents();
    griddep_wait();
    if ((int)blockIdx.x < tiles) {
        const int tile = (int)blockIdx.x;
        long long row0, end;
        if (a.offsets) {
            // the last group whose first tile is not past this one; in bounds whatever the offsets hold
            int n = 0;
            for (int i = lane + 1; i <= a.groups; i += 32) n += (min(max(__ldg(a.offsets + i), 0), a.M) >> 7) + i <= tile ? 1 : 0;
            const int g = __reduce_add_sync(kAll, n);
            const int start = min(max(__ldg(a.offsets + g), 0), a.M), local = tile - (start >> 7) - g;
            if (local < 0) return;  // before the first group: no row's place
            row0 = start + local * 128LL;
            end = g < a.groups ? min(max(__ldg(a.offsets + g + 1), 0), a.M) : a.M;
        } else {
            const int g = tile / a.tiles_per;
            row0 = (long long)g * a.per + (long long)(tile - g * a.tiles_per) * 128;
            end = (long long)(g + 1) * a.per;
        }
        if (row0 >= end) return;
        const uint32_t *from[4];
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long m = row0 + lane + 32 * i;
            in[i] = m < end;
            int src = in[i] ? __ldg(a.rows + m) : 0;
            if (src < 0 || src >= a.x_rows) src = 0;  // reported where the codes are copied
            from[i] = work_scales + (size_t)src * chunks;
        }
        uint8_t *to = a.scales + (size_t)tile * chunks * 512 + lane * 16;
        for (unsigned c = warp; c < chunks; c += kRowWarps) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = in[i] ? __ldg(from[i] + c) : 0u;
            if (in[3])
                *reinterpret_cast<uint4 *>(to + (size_t)c * 512) = make_uint4(v[0], v[1], v[2], v[3]);
            else
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (in[i]) *reinterpret_cast<uint32_t *>(to + (size_t)c * 512 + 4 * i) = v[i];
        }
        return;
    }
    const long long m = (long long)(blockIdx.x - tiles) * kRowWarps + warp;
    if (m >= a.M) return;
    long long src = __ldg(a.rows + m);
    if (src < 0 || src >= a.x_rows) {
        if (lane == 0) atomicOr(a.err, BN_DEVERR_PERM_RANGE);
        src = 0;
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(work + src * (a.K / 2));
    uint4 *to = reinterpret_cast<uint4 *>(a.data + m * (a.K / 2));
    const unsigned n = (unsigned)a.K / 32;
    constexpr unsigned kAhead = 4;
    for (unsigned i = lane; i < n; i += 32 * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u)
            if (i + 32 * u < n) v[u] = __ldg(from + i + 32 * u);
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u)
            if (i + 32 * u < n) to[i + 32 * u] = v[u];
    }
}

// Eight values at an address of 16 bytes' alignment.
template <typename T> __device__ __forceinline__ void store8(T *out, const f2 *v);
template <> __device__ __forceinline__ void store8(float *out, const f2 *v)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(v[i], x[2 * i], x[2 * i + 1]);
    reinterpret_cast<float4 *>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <> __device__ __forceinline__ void store8(__nv_bfloat16 *out, const f2 *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = round2(v[i]);
    *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ void store8(__half *out, const f2 *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x, y;
        f2_split(v[i], x, y);
        const __half2 h = __floats2half2_rn(x, y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool MX>
__global__ void __launch_bounds__(kRowWarps * 32) dequantize_kernel(const __grid_constant__ QuantArgs a, int chunks, int share)
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
    constexpr unsigned kChunk = MX ? 128 : 64;
    constexpr unsigned kAhead = 4;  // steps of 256 values, 8 a lane, whose loads are in flight together
    const unsigned k1 = min((unsigned)a.K, (blockIdx.y + 1) * (unsigned)share);
    unsigned k = blockIdx.y * (unsigned)share + lane * 8u;
    if (!p.in) {  // no group, no scales
        const f2 zeros[4] = {};
        for (; k < k1; k += 256) store8<T>(out + k, zeros);
        return;
    }
    const auto steps = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        uint32_t q[kAhead], b[kAhead];
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u) {
            const unsigned at = k + 256 * u;
            if (FULL || at < k1) {
                q[u] = __ldg(reinterpret_cast<const uint32_t *>(data + at / 2));
                b[u] = __ldg(scales + (size_t)(at / kChunk) * 512 + at % kChunk / (MX ? 32 : 16));
            }
        }
#pragma unroll
        for (unsigned u = 0; u < kAhead; ++u) {
            const unsigned at = k + 256 * u;
            if (!FULL && at >= k1) break;
            const float s = (MX ? e8m0_value(b[u]) : e4m3_value(b[u])) * a.tensor_scale;
            const f2 s2 = f2_make(s, s);
            uint32_t h[4];
            asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(q[u]));
            f2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                v[i] = mul2(f2_make(f.x, f.y), s2);
            }
            store8<T>(out + at, v);
        }
        k += 256 * kAhead;
    };
    while (k - lane * 8u + 256 * kAhead <= k1) steps(std::true_type{});
    while (k < k1) steps(std::false_type{});
}

// Values of a row per block: whole rows when there are warps enough for the
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
    const int per = fmt ? 128 : 64, chunks = (a.K + per - 1) / per;
    if (!a.work) {
        split_rows(a, sms, &grid, &share);
        auto *k = dtype == 0 ? (fmt ? quantize_kernel<__nv_bfloat16, true, false> : quantize_kernel<__nv_bfloat16, false, false>)
                             : (fmt ? quantize_kernel<__half, true, false> : quantize_kernel<__half, false, false>);
        return launch_kernel(k, grid, dim3(kRowWarps * 32), 0, pdl, 1, st, a, chunks, share);
    }
    QuantArgs once = a;
    once.rows = nullptr;
    once.M = (int)a.x_rows;
    once.data = a.work;
    once.scales = a.work + (size_t)a.x_rows * (a.K / 2);
    split_rows(once, sms, &grid, &share);
    auto *k = dtype == 0 ? (fmt ? quantize_kernel<__nv_bfloat16, true, true> : quantize_kernel<__nv_bfloat16, false, true>)
                         : (fmt ? quantize_kernel<__half, true, true> : quantize_kernel<__half, false, true>);
    const cudaError_t e = launch_kernel(k, grid, dim3(kRowWarps * 32), 0, pdl, 1, st, once, chunks, share);
    if (e != cudaSuccess) return e;
    const int tiles = a.offsets ? a.M / 128 + a.groups + 1 : a.groups * a.tiles_per;
    return launch_kernel(place_rows_kernel, dim3((unsigned)(tiles + (a.M + kRowWarps - 1) / kRowWarps)),
                         dim3(kRowWarps * 32), 0, pdl, 1, st, a, (const uint8_t *)a.work, (const uint32_t *)once.scales,
                         (unsigned)chunks, tiles);
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
