// bn_experts_abi.cu -- the C entry points around the experts: host-side
// validation and launches.  Like the rest of the ABI, arguments are checked
// before any CUDA call, and each call enqueues one kernel (two for a call that
// goes through a workspace) or nothing.
#include <cmath>

#include <cuda_runtime.h>

#include "../../include/beamnorm.h"
#include "bn_experts.h"
#include "bn_host.h"
#include "bn_internal.h"

namespace bn {
namespace {

// Rows and slots are counted in int32, rounded up to tiles and blocks.
constexpr long long kMaxRows = (1LL << 31) - 1024;
constexpr int kMaxInt8K = 131056;
constexpr int kNominalSms = 152;  // of a GB300, where no device is asked

size_t dtype_size(int dtype) { return dtype == BN_FP32 ? 4 : 2; }

bn_status check_dtype(int dtype, bool fp32)
{
    BN_REQUIRE(dtype == BN_BF16 || dtype == BN_FP16 || (fp32 && dtype == BN_FP32), "dtype %d is not served here", dtype);
    return BN_OK;
}

bn_status check_route(int dtype, long long ld, int T, int E, int k, int R, int score)
{
    BN_TRY(check_dtype(dtype, true));
    BN_REQUIRE(T >= 0, "T=%d is negative", T);
    BN_REQUIRE(E >= 1, "E=%d is not positive", E);
    BN_REQUIRE(k >= 1 && k <= kMaxK, "k=%d outside [1, %d]", k, kMaxK);
    BN_REQUIRE(k <= E, "k=%d above E=%d", k, E);
    BN_REQUIRE(R >= 1 && R <= kMaxR, "R=%d outside [1, %d]", R, kMaxR);
    BN_REQUIRE(ld >= E, "ld=%lld below E=%d", ld, E);
    BN_REQUIRE(score == BN_SCORE_SOFTMAX || score == BN_SCORE_SIGMOID, "score %d is unknown", score);
    if (E > kMaxExperts) return fail(BN_ERR_UNSUPPORTED, "E=%d above the served maximum %d", E, kMaxExperts);
    if ((long long)T * k > kMaxRows)
        return fail(BN_ERR_UNSUPPORTED, "T*k=%lld does not fit int32 slot indices", (long long)T * k);
    return BN_OK;
}

bn_status check_element(const void *p, size_t size, const char *name)
{
    BN_REQUIRE(p, "%s is NULL", name);
    BN_REQUIRE(aligned(p, size), "%s is not %d-byte aligned", name, (int)size);
    return BN_OK;
}

// The bytes that T rows of E elements, ld apart, span.
size_t span(int T, long long ld, int E, size_t size) { return T ? ((size_t)(T - 1) * (size_t)ld + (size_t)E) * size : 0; }

// 16-byte vectors fit every row.
bool vectors(const void *p, long long ld, int E, size_t size)
{
    const long long per = 16 / (long long)size;
    return aligned(p, 16) && ld % per == 0 && E % per == 0;
}

bn_status check_power_of_two(float v)
{
    int e;
    BN_REQUIRE(std::isfinite(v) && v > 0.0f && std::frexp(v, &e) == 0.5f && e >= -63 && e <= 65,
               "tensor_scale must be a power of two in [2^-64, 2^64]");
    return BN_OK;
}

long long scale_tiles(long long M, int groups, bool ragged)
{
    if (ragged) return M / 128 + groups + 1;
    const long long per = M / groups;
    return groups * ((per + 127) / 128);
}

size_t scale_bytes(long long M, int K, int groups, bool ragged, int fmt)
{
    const int per = fmt == BN_MXFP4 ? 128 : 64;
    return (size_t)scale_tiles(M, groups, ragged) * (size_t)((K + per - 1) / per) * 512;
}

bn_status check_fp4(int fmt, int M, int K, int groups, const int32_t *offsets)
{
    BN_REQUIRE(fmt == BN_NVFP4 || fmt == BN_MXFP4, "format %d is unknown", fmt);
    BN_REQUIRE(M >= 0, "M=%d is negative", M);
    BN_REQUIRE(K >= 32 && K % 32 == 0, "K=%d is not a positive multiple of 32", K);
    BN_REQUIRE(groups >= 1, "groups=%d is not positive", groups);
    BN_REQUIRE(offsets || M % groups == 0, "M=%d rows do not make %d equal groups", M, groups);
    BN_REQUIRE(aligned(offsets, 4), "offsets is not 4-byte aligned");
    if (offsets && groups > kMaxExperts)
        return fail(BN_ERR_UNSUPPORTED, "groups=%d above the served maximum %d", groups, kMaxExperts);
    if (M > kMaxRows) return fail(BN_ERR_UNSUPPORTED, "M=%d above the served maximum %lld", M, kMaxRows);
    if (K > (1 << 20)) return fail(BN_ERR_UNSUPPORTED, "K=%d above the served maximum %d", K, 1 << 20);
    return BN_OK;
}

bn_status launched(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return BN_OK;
    (void)cudaGetLastError();  // a failed launch leaves no error behind for the caller's next call
    return cuda_fail(e, what);
}

// What the three products of a linear layer share.
bn_status check_linear(int dtype, int M, int E, int N, int K, const int32_t *offsets)
{
    BN_TRY(check_dtype(dtype, false));
    BN_REQUIRE(M >= 0, "M=%d is negative", M);
    BN_REQUIRE(E >= 1, "E=%d is not positive", E);
    BN_REQUIRE(N >= 8 && N % 8 == 0, "N=%d is not a positive multiple of 8", N);
    BN_REQUIRE(K >= 8 && K % 8 == 0, "K=%d is not a positive multiple of 8", K);
    BN_REQUIRE(offsets || E == 1, "offsets is NULL with E=%d experts", E);
    BN_REQUIRE(aligned(offsets, 4), "offsets is not 4-byte aligned");
    if (E > kMaxExperts) return fail(BN_ERR_UNSUPPORTED, "E=%d above the served maximum %d", E, kMaxExperts);
    if (M > kMaxRows) return fail(BN_ERR_UNSUPPORTED, "M=%d above the served maximum %lld", M, kMaxRows);
    if (N > (1 << 20) || K > (1 << 20))
        return fail(BN_ERR_UNSUPPORTED, "N=%d, K=%d: above the served maximum %d", N, K, 1 << 20);
    if ((long long)N * K > (1LL << 37))  // an expert's bytes in a tensor map
        return fail(BN_ERR_UNSUPPORTED, "N * K=%lld above the served maximum %lld", (long long)N * K, 1LL << 37);
    return BN_OK;
}

bn_status check_rows(const void *p, const char *name, long long ld, int width)
{
    BN_REQUIRE(ld >= width && ld % 8 == 0, "%s: ld=%lld is not a multiple of 8 of at least %d", name, ld, width);
    if (ld > (1LL << 36)) return fail(BN_ERR_UNSUPPORTED, "%s: ld=%lld above the served maximum", name, ld);
    return check_ptr16(p, name);
}

bn_status check_int8(int M, int K)
{
    BN_REQUIRE(M >= 0, "M=%d is negative", M);
    BN_REQUIRE(K >= 16 && K % 16 == 0, "K=%d is not a positive multiple of 16", K);
    if (M > kMaxRows) return fail(BN_ERR_UNSUPPORTED, "M=%d above the served maximum %lld", M, kMaxRows);
    // K products of two codes of at most 128 each fit 32 bits
    if (K > kMaxInt8K) return fail(BN_ERR_UNSUPPORTED, "K=%d above the served maximum %d", K, kMaxInt8K);
    return BN_OK;
}

bn_status check_swiglu(int dtype, int M, int F, long long ld)
{
    BN_TRY(check_dtype(dtype, true));
    BN_REQUIRE(M >= 0, "M=%d is negative", M);
    BN_REQUIRE(F >= 1, "F=%d is not positive", F);
    BN_REQUIRE(ld >= 2LL * F, "ld=%lld below 2 * F=%lld", ld, 2LL * F);
    if (M > kMaxRows) return fail(BN_ERR_UNSUPPORTED, "M=%d above the served maximum %lld", M, kMaxRows);
    if (F > (1 << 28)) return fail(BN_ERR_UNSUPPORTED, "F=%d above the served maximum %d", F, 1 << 28);
    return BN_OK;
}

// With a workspace of enough bytes, rows by index go to their places there first; x, ld and the
// arguments' rows are then those of the workspace.
bn_status place_rows(LinearArgs &a, const void *&x, long long &ld, int K, void *workspace, size_t bytes, const DeviceInfo &d,
                     void *stream)
{
    const size_t need = a.rows ? bn_expert_linear_workspace_bytes(a.M, K) : 0;
    if (need == 0 || !workspace || bytes < need) return BN_OK;
    BN_TRY(launched(launch_place_rows(x, ld, a.x_rows, a.rows, a.M, a.offsets, a.E, K, workspace, nullptr, nullptr, d.err, d.sms,
                                      dependent_launch(), (cudaStream_t)stream),
                    "launching place_rows"));
    x = workspace;
    ld = K;
    a.rows = nullptr;
    a.x_rows = a.M;
    return BN_OK;
}

LinearArgs linear_args(int dtype, int M, int E, int F, int D, int K, const int32_t *offsets, void *out, unsigned *err)
{
    LinearArgs a = {};
    a.M = M;
    a.E = E;
    a.F = F;
    a.D = D;
    a.K = K;
    a.offsets = offsets;
    a.out = out;
    a.dtype = dtype;
    a.err = err;
    return a;
}

}  // namespace
}  // namespace bn

using namespace bn;

extern "C" {

bn_status bn_route(const void *logits, bn_dtype dtype, long long ld, int T, int E, int k, const float *bias,
                   bn_score score, int groups, int top_groups, int group_top, int renormalize, float scale, int R,
                   int32_t *ids, float *w, void *stream)
{
    clear_message();
    BN_TRY(check_route(dtype, ld, T, E, k, R, score));
    BN_REQUIRE(groups >= 1 && E % groups == 0, "E=%d experts do not make groups=%d equal groups", E, groups);
    BN_REQUIRE(top_groups >= 1 && top_groups <= groups, "top_groups=%d outside [1, groups=%d]", top_groups, groups);
    BN_REQUIRE(group_top == 1 || group_top == 2, "group_top=%d is neither 1 nor 2", group_top);
    BN_REQUIRE(std::isfinite(scale), "scale must be finite");
    BN_REQUIRE((long long)top_groups * (E / groups) >= k, "k=%d above the %d experts of top_groups=%d groups", k,
               top_groups * (E / groups), top_groups);
    if (groups > kMaxGroups)
        return fail(BN_ERR_UNSUPPORTED, "groups=%d above the served maximum %d", groups, kMaxGroups);
    if (T == 0) return BN_OK;
    BN_TRY(check_element(logits, dtype_size(dtype), "logits"));
    BN_REQUIRE(aligned(bias, 4), "bias is not 4-byte aligned");
    BN_TRY(check_ptr4(ids, "ids"));
    BN_TRY(check_ptr4(w, "w"));
    const Range writes[] = {{ids, (size_t)T * k * 4, "ids"}, {w, (size_t)R * T * k * 4, "w"}};
    const Range reads[] = {{logits, span(T, ld, E, dtype_size(dtype)), "logits"}, {bias, (size_t)E * 4, "bias"}};
    BN_TRY(check_overlaps(writes, 2, reads, 2));
    RouteArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.E = E;
    a.k = k;
    a.bias = bias;
    a.sigmoid = score == BN_SCORE_SIGMOID;
    a.groups = top_groups == groups ? 1 : groups;  // every group stays: none are ranked
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.R = R;
    a.ids = ids;
    a.w = w;
    a.vec = vectors(logits, ld, E, dtype_size(dtype));
    a.bias_vec = vectors(bias, 4, E, 4);
    return launched(launch_route(a, dtype, dependent_launch(), (cudaStream_t)stream), "launching route");
}

bn_status bn_route_backward(const void *logits, bn_dtype dtype, long long ld, int T, int E, int k, const int32_t *ids,
                            const float *dw, int R, bn_score score, int renormalize, float scale, void *dlogits,
                            void *stream)
{
    clear_message();
    BN_TRY(check_route(dtype, ld, T, E, k, R, score));
    BN_REQUIRE(std::isfinite(scale), "scale must be finite");
    if (T == 0) return BN_OK;
    const size_t size = dtype_size(dtype);
    BN_TRY(check_element(logits, size, "logits"));
    BN_TRY(check_ptr4(ids, "ids"));
    BN_TRY(check_ptr4(dw, "dw"));
    BN_TRY(check_element(dlogits, size, "dlogits"));
    const Range writes[] = {{dlogits, (size_t)T * E * size, "dlogits"}};
    const Range reads[] = {{logits, span(T, ld, E, size), "logits"},
                           {ids, (size_t)T * k * 4, "ids"},
                           {dw, (size_t)R * T * k * 4, "dw"}};
    BN_TRY(check_overlaps(writes, 1, reads, 3));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    RouteBackwardArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.E = E;
    a.k = k;
    a.ids = ids;
    a.dw = dw;
    a.R = R;
    a.sigmoid = score == BN_SCORE_SIGMOID;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.dlogits = dlogits;
    a.err = d->err;
    a.vec = vectors(logits, ld, E, size) && vectors(dlogits, E, E, size);
    return launched(launch_route_backward(a, dtype, dependent_launch(), (cudaStream_t)stream),
                    "launching route_backward");
}

bn_status bn_expert_plan(const int32_t *ids, int T, int k, int E, int R, int32_t *perm, int32_t *offsets,
                         int32_t *rows, void *stream)
{
    clear_message();
    BN_REQUIRE(T >= 0, "T=%d is negative", T);
    BN_REQUIRE(E >= 1, "E=%d is not positive", E);
    BN_REQUIRE(k >= 1 && k <= kMaxK, "k=%d outside [1, %d]", k, kMaxK);
    BN_REQUIRE(R >= 1 && R <= kMaxR, "R=%d outside [1, %d]", R, kMaxR);
    if (E > kMaxExperts) return fail(BN_ERR_UNSUPPORTED, "E=%d above the served maximum %d", E, kMaxExperts);
    if ((long long)T * k > kMaxRows)
        return fail(BN_ERR_UNSUPPORTED, "T*k=%lld does not fit int32 slot indices", (long long)T * k);
    BN_TRY(check_ptr4(offsets, "offsets"));
    if (T > 0) {
        BN_TRY(check_ptr4(ids, "ids"));
        BN_TRY(check_ptr4(perm, "perm"));
        BN_TRY(check_ptr4(rows, "rows"));
    }
    const size_t n = (size_t)T * k * 4;
    const Range writes[] = {{perm, n * R, "perm"}, {offsets, (size_t)(E + 1) * 4, "offsets"}, {rows, n, "rows"}};
    const Range reads[] = {{ids, n, "ids"}};
    BN_TRY(check_overlaps(writes, 3, reads, 1));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    PlanArgs a = {};
    a.ids = ids;
    a.slots = T * k;
    a.k = k;
    a.E = E;
    a.R = R;
    a.perm = perm;
    a.offsets = offsets;
    a.rows = rows;
    a.err = d->err;
    return launched(launch_plan(a, dependent_launch(), (cudaStream_t)stream), "launching expert_plan");
}

size_t bn_fp4_scale_bytes(int M, int K, int groups, int ragged, bn_fp4 format)
{
    if (M < 0 || K < 32 || K % 32 != 0 || groups < 1 || (!ragged && M % groups != 0)) return 0;
    if (format != BN_NVFP4 && format != BN_MXFP4) return 0;
    return scale_bytes(M, K, groups, ragged != 0, format);
}

size_t bn_quantize_fp4_workspace_bytes(int x_rows, int M, int K, bn_fp4 format)
{
    if (x_rows < 1 || M < 1 || K < 32 || K % 32 != 0 || (format != BN_NVFP4 && format != BN_MXFP4)) return 0;
    // What is saved is the quantisation of M - x_rows rows; what it costs is a second kernel whose
    // scale tiles take 10 us and more where they are few.  Measured over 316 shapes of 300 to 5000
    // rows taken 4 to 50 times, K from 544 to 8192, both formats: at most 13 % slower where taken
    // (16384 places of 2048 rows of 1024 values, MXFP4: 8.0 us, place by place 7.1), at most 21 %
    // left where not (8000 of 1000 rows of 5120: 11.7 us, 9.7 this way).
    const long long repeats = (long long)M - x_rows, work = (long long)M * K;
    if (repeats < 9000 || M / 4 < x_rows || work < (1LL << 24)) return 0;
    if (M / 8 < x_rows && work < (1LL << 25)) return 0;
    const int per = format == BN_MXFP4 ? 128 : 64;
    return (size_t)x_rows * ((size_t)K / 2 + 4 * (size_t)((K + per - 1) / per));
}

bn_status bn_quantize_fp4(const void *x, bn_dtype dtype, long long ld, int x_rows, const int32_t *rows, int M, int K,
                          const int32_t *offsets, int groups, bn_fp4 format, float tensor_scale, uint8_t *data,
                          uint8_t *scales, void *workspace, size_t workspace_bytes, void *stream)
{
    clear_message();
    BN_TRY(check_dtype(dtype, false));
    BN_TRY(check_fp4(format, M, K, groups, offsets));
    BN_TRY(check_power_of_two(tensor_scale));
    BN_REQUIRE(ld >= K && ld % 8 == 0, "ld=%lld is not a multiple of 8 of at least K=%d", ld, K);
    BN_REQUIRE(x_rows >= 0, "x_rows=%d is negative", x_rows);
    BN_REQUIRE(rows || x_rows == M, "x has %d rows, M=%d are wanted and no rows are given", x_rows, M);
    if (M == 0) return BN_OK;
    BN_REQUIRE(x_rows > 0, "x has no rows");
    BN_TRY(check_ptr16(x, "x"));
    BN_REQUIRE(aligned(rows, 4), "rows is not 4-byte aligned");
    BN_TRY(check_ptr16(data, "data"));
    BN_TRY(check_ptr16(scales, "scales"));
    BN_TRY(check_ptr16(workspace, "workspace", false));
    const Range writes[] = {{data, (size_t)M * (K / 2), "data"},
                            {scales, scale_bytes(M, K, groups, offsets != nullptr, format), "scales"},
                            {workspace, workspace_bytes, "workspace"}};
    const Range reads[] = {{x, span(x_rows, ld, K, 2), "x"},
                           {rows, (size_t)M * 4, "rows"},
                           {offsets, (size_t)(groups + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 3, reads, 3));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    const size_t need = rows ? bn_quantize_fp4_workspace_bytes(x_rows, M, K, format) : 0;
    QuantArgs a = {};
    a.work = need && workspace && workspace_bytes >= need ? static_cast<uint8_t *>(workspace) : nullptr;
    a.x = x;
    a.ld = ld;
    a.x_rows = x_rows;
    a.rows = rows;
    a.M = M;
    a.K = K;
    a.offsets = offsets;
    a.groups = groups;
    a.per = M / groups;
    a.tiles_per = (a.per + 127) / 128;
    a.tensor_scale = tensor_scale;
    a.inv_tensor_scale = 1.0f / tensor_scale;
    a.data = data;
    a.scales = scales;
    a.err = d->err;
    return launched(launch_quantize(a, dtype, format, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching quantize_fp4");
}

bn_status bn_dequantize_fp4(const uint8_t *data, const uint8_t *scales, int M, int K, const int32_t *offsets,
                            int groups, bn_fp4 format, float tensor_scale, void *out, bn_dtype dtype, void *stream)
{
    clear_message();
    BN_TRY(check_dtype(dtype, true));
    BN_TRY(check_fp4(format, M, K, groups, offsets));
    BN_TRY(check_power_of_two(tensor_scale));
    if (M == 0) return BN_OK;
    BN_TRY(check_ptr16(data, "data"));
    BN_TRY(check_ptr16(scales, "scales"));
    BN_TRY(check_ptr16(out, "out"));
    const Range writes[] = {{out, (size_t)M * K * dtype_size(dtype), "out"}};
    const Range reads[] = {{data, (size_t)M * (K / 2), "data"},
                           {scales, scale_bytes(M, K, groups, offsets != nullptr, format), "scales"},
                           {offsets, (size_t)(groups + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 1, reads, 3));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    QuantArgs a = {};
    a.M = M;
    a.K = K;
    a.offsets = offsets;
    a.groups = groups;
    a.per = M / groups;
    a.tiles_per = (a.per + 127) / 128;
    a.tensor_scale = tensor_scale;
    a.data = const_cast<uint8_t *>(data);
    a.scales = const_cast<uint8_t *>(scales);
    a.out = out;
    a.err = d->err;
    return launched(launch_dequantize(a, dtype, format, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching dequantize_fp4");
}

bn_status bn_expert_product(const uint8_t *a, const uint8_t *a_scales, int M, const uint8_t *w,
                            const uint8_t *w_scales, int E, int N, int K, const int32_t *offsets, bn_fp4 format,
                            float alpha, uint16_t *out, void *stream)
{
    clear_message();
    BN_TRY(check_fp4(format, M, K, 1, nullptr));
    BN_REQUIRE(E >= 1, "E=%d is not positive", E);
    BN_REQUIRE(N >= 8 && N % 8 == 0, "N=%d is not a positive multiple of 8", N);
    BN_REQUIRE(offsets || E == 1, "offsets is NULL with E=%d experts", E);
    BN_REQUIRE(aligned(offsets, 4), "offsets is not 4-byte aligned");
    BN_REQUIRE(std::isfinite(alpha), "alpha must be finite");
    if (E > kMaxExperts) return fail(BN_ERR_UNSUPPORTED, "E=%d above the served maximum %d", E, kMaxExperts);
    if ((long long)E * N >= (1LL << 31))
        return fail(BN_ERR_UNSUPPORTED, "E*N=%lld weight rows do not fit int32", (long long)E * N);
    const int chunks = (K + (format == BN_MXFP4 ? 127 : 63)) / (format == BN_MXFP4 ? 128 : 64);
    const long long a_tiles = scale_tiles(M, E, offsets != nullptr), w_tiles = (long long)E * ((N + 127) / 128);
    if ((a_tiles > w_tiles ? a_tiles : w_tiles) * chunks >= (1LL << 31))
        return fail(BN_ERR_UNSUPPORTED, "M=%d, E=%d, N=%d, K=%d: the scale tiles do not fit int32", M, E, N, K);
    if (M == 0) return BN_OK;
    BN_TRY(check_ptr16(a, "a"));
    BN_TRY(check_ptr16(a_scales, "a_scales"));
    BN_TRY(check_ptr16(w, "w"));
    BN_TRY(check_ptr16(w_scales, "w_scales"));
    BN_TRY(check_ptr16(out, "out"));
    const Range writes[] = {{out, (size_t)M * N * 2, "out"}};
    const Range reads[] = {{a, (size_t)M * (K / 2), "a"},
                           {a_scales, scale_bytes(M, K, E, offsets != nullptr, format), "a_scales"},
                           {w, (size_t)E * N * (K / 2), "w"},
                           {w_scales, (size_t)E * scale_bytes(N, K, 1, false, format), "w_scales"},
                           {offsets, (size_t)(E + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 1, reads, 5));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    ProductArgs p = {};
    p.M = M;
    p.E = E;
    p.N = N;
    p.K = K;
    p.offsets = offsets;
    p.a_scales = a_scales;
    p.a_tiles = a_tiles;
    p.w_scales = w_scales;
    p.chunks = chunks;
    p.alpha = alpha;
    p.out = out;
    p.err = d->err;
    return launched(launch_product(p, a, w, format, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching expert_product");
}

size_t bn_expert_linear_workspace_bytes(int M, int K)
{
    // Fetching a row by its index costs the copying thread about 25 cycles for every 64 values, which
    // the stream of weights hides up to about 30 rows of a group: with no more rows than that in
    // all, none go through the workspace.
    return M > 32 && K >= 8 && K % 8 == 0 ? (size_t)M * K * 2 : 0;
}

bn_status bn_expert_linear(const void *x, bn_dtype dtype, long long ld, int x_rows, const int32_t *rows, int M,
                           const void *w, int E, int N, int K, const int32_t *offsets, void *y, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    clear_message();
    BN_TRY(check_linear(dtype, M, E, N, K, offsets));
    BN_REQUIRE(x_rows >= 0, "x_rows=%d is negative", x_rows);
    BN_REQUIRE(rows || x_rows == M, "x has %d rows, M=%d are wanted and no rows are given", x_rows, M);
    if (M == 0) return BN_OK;
    BN_REQUIRE(x_rows > 0, "x has no rows");
    BN_REQUIRE(aligned(rows, 4), "rows is not 4-byte aligned");
    BN_TRY(check_rows(x, "x", ld, K));
    BN_TRY(check_ptr16(w, "w"));
    BN_TRY(check_ptr16(y, "y"));
    BN_TRY(check_ptr16(workspace, "workspace", false));
    const Range writes[] = {{y, (size_t)M * N * 2, "y"}, {workspace, workspace_bytes, "workspace"}};
    const Range reads[] = {{x, span(x_rows, ld, K, 2), "x"},
                           {rows, (size_t)M * 4, "rows"},
                           {w, (size_t)E * N * K * 2, "w"},
                           {offsets, (size_t)(E + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 2, reads, 4));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    LinearArgs a = linear_args(dtype, M, E, N, K, 0, offsets, y, d->err);
    a.rows = rows;
    a.x_rows = x_rows;
    BN_TRY(place_rows(a, x, ld, K, workspace, workspace_bytes, *d, stream));
    return launched(launch_linear(a, kForward, x, ld, w, 0, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching expert_linear");
}

bn_status bn_expert_linear_dx(const void *dy, bn_dtype dtype, long long ld_dy, int M, const void *w, int E, int N, int K,
                              const int32_t *offsets, void *dx, void *stream)
{
    clear_message();
    BN_TRY(check_linear(dtype, M, E, N, K, offsets));
    if (M == 0) return BN_OK;
    BN_TRY(check_rows(dy, "dy", ld_dy, N));
    BN_TRY(check_ptr16(w, "w"));
    BN_TRY(check_ptr16(dx, "dx"));
    const Range writes[] = {{dx, (size_t)M * K * 2, "dx"}};
    const Range reads[] = {{dy, span(M, ld_dy, N, 2), "dy"},
                           {w, (size_t)E * N * K * 2, "w"},
                           {offsets, (size_t)(E + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 1, reads, 3));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    const LinearArgs a = linear_args(dtype, M, E, K, N, 0, offsets, dx, d->err);
    return launched(launch_linear(a, kInputGrad, dy, ld_dy, w, 0, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching expert_linear_dx");
}

bn_status bn_expert_linear_dw(const void *dy, bn_dtype dtype, long long ld_dy, int M, const void *x, long long ld,
                              int x_rows, const int32_t *rows, int E, int N, int K, const int32_t *offsets, void *dw,
                              bn_dtype dw_dtype, int accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    clear_message();
    BN_TRY(check_linear(dtype, M, E, N, K, offsets));
    BN_REQUIRE(dw_dtype == dtype || dw_dtype == BN_FP32, "dw_dtype %d is neither dtype nor BN_FP32", (int)dw_dtype);
    BN_REQUIRE(!accumulate || dw_dtype == BN_FP32, "accumulate takes BN_FP32 gradients");
    BN_REQUIRE(x_rows >= 0, "x_rows=%d is negative", x_rows);
    BN_REQUIRE(rows || x_rows == M, "x has %d rows, M=%d are wanted and no rows are given", x_rows, M);
    BN_TRY(check_ptr16(dw, "dw"));
    const size_t bytes = (size_t)E * N * K * dtype_size(dw_dtype);
    if (M == 0) {  // every group is empty
        if (accumulate) return BN_OK;
        return launched(cudaMemsetAsync(dw, 0, bytes, (cudaStream_t)stream), "clearing dw");
    }
    BN_REQUIRE(x_rows > 0, "x has no rows");
    BN_REQUIRE(aligned(rows, 4), "rows is not 4-byte aligned");
    BN_TRY(check_rows(dy, "dy", ld_dy, N));
    BN_TRY(check_rows(x, "x", ld, K));
    BN_TRY(check_ptr16(workspace, "workspace", false));
    const Range writes[] = {{dw, bytes, "dw"}, {workspace, workspace_bytes, "workspace"}};
    const Range reads[] = {{dy, span(M, ld_dy, N, 2), "dy"},
                           {x, span(x_rows, ld, K, 2), "x"},
                           {rows, (size_t)M * 4, "rows"},
                           {offsets, (size_t)(E + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 2, reads, 4));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    LinearArgs a = linear_args(dtype, M, E, N, 0, K, offsets, dw, d->err);
    a.rows = rows;
    a.x_rows = x_rows;
    a.out_fp32 = dw_dtype == BN_FP32;
    a.accumulate = accumulate != 0;
    BN_TRY(place_rows(a, x, ld, K, workspace, workspace_bytes, *d, stream));
    return launched(launch_linear(a, kWeightGrad, x, ld, dy, ld_dy, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching expert_linear_dw");
}

bn_status bn_swiglu(const void *x, bn_dtype dtype, long long ld, int M, int F, void *y, void *stream)
{
    clear_message();
    BN_TRY(check_swiglu(dtype, M, F, ld));
    if (M == 0) return BN_OK;
    const size_t size = dtype_size(dtype);
    BN_TRY(check_element(x, size, "x"));
    BN_TRY(check_element(y, size, "y"));
    const Range writes[] = {{y, (size_t)M * F * size, "y"}};
    const Range reads[] = {{x, span(M, ld, 2 * F, size), "x"}};
    BN_TRY(check_overlaps(writes, 1, reads, 1));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    SwigluArgs a = {};
    a.x = x;
    a.out = y;
    a.ld = ld;
    a.M = M;
    a.F = F;
    a.vec = vectors(x, ld, F, size) && vectors(y, F, F, size);
    return launched(launch_swiglu(a, dtype, false, d->sms, dependent_launch(), (cudaStream_t)stream), "launching swiglu");
}

bn_status bn_swiglu_backward(const void *x, bn_dtype dtype, long long ld, int M, int F, const void *dy, long long ld_dy,
                             void *dx, void *stream)
{
    clear_message();
    BN_TRY(check_swiglu(dtype, M, F, ld));
    BN_REQUIRE(ld_dy >= F, "ld_dy=%lld below F=%d", ld_dy, F);
    if (M == 0) return BN_OK;
    const size_t size = dtype_size(dtype);
    BN_TRY(check_element(x, size, "x"));
    BN_TRY(check_element(dy, size, "dy"));
    BN_TRY(check_element(dx, size, "dx"));
    const Range writes[] = {{dx, (size_t)M * 2 * F * size, "dx"}};
    const Range reads[] = {{x, span(M, ld, 2 * F, size), "x"}, {dy, span(M, ld_dy, F, size), "dy"}};
    BN_TRY(check_overlaps(writes, 1, reads, 2));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    SwigluArgs a = {};
    a.x = x;
    a.dy = dy;
    a.out = dx;
    a.ld = ld;
    a.ld_dy = ld_dy;
    a.M = M;
    a.F = F;
    a.vec = vectors(x, ld, F, size) && vectors(dy, ld_dy, F, size) && vectors(dx, F, F, size);
    return launched(launch_swiglu(a, dtype, true, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching swiglu_backward");
}

size_t bn_quantize_int8_workspace_bytes(int x_rows, int M, int K)
{
    if (x_rows < 1 || M < 1 || K < 16 || K % 16 != 0) return 0;
    // What is saved is the quantisation of the repeats; what it costs is a second kernel.  Measured,
    // place by place / through the workspace (us): 4096 rows of 5120 taken 8 times 80 / 49, 4 times
    // 45 / 35, twice 27 / 27; 1000 of 8192 10 times 39 / 27; 500 of 4096 16 times 20 / 16; 300 of
    // 5120 8 times 12 / 12.
    const long long repeats = (long long)M - x_rows;
    if (M / 2 < x_rows || repeats * K < (1LL << 24)) return 0;
    return (size_t)x_rows * ((size_t)K + 4);
}

bn_status bn_quantize_int8(const void *x, bn_dtype dtype, long long ld, int x_rows, const int32_t *rows, int M, int K,
                           int8_t *data, float *scales, void *workspace, size_t workspace_bytes, void *stream)
{
    clear_message();
    BN_TRY(check_dtype(dtype, true));
    BN_TRY(check_int8(M, K));
    const size_t size = dtype_size(dtype);
    const int per = 16 / (int)size;
    BN_REQUIRE(ld >= K && ld % per == 0, "ld=%lld is not a multiple of %d of at least K=%d", ld, per, K);
    BN_REQUIRE(x_rows >= 0, "x_rows=%d is negative", x_rows);
    BN_REQUIRE(rows || x_rows == M, "x has %d rows, M=%d are wanted and no rows are given", x_rows, M);
    if (M == 0) return BN_OK;
    BN_REQUIRE(x_rows > 0, "x has no rows");
    BN_TRY(check_ptr16(x, "x"));
    BN_REQUIRE(aligned(rows, 4), "rows is not 4-byte aligned");
    BN_TRY(check_ptr16(data, "data"));
    BN_TRY(check_ptr4(scales, "scales"));
    BN_TRY(check_ptr16(workspace, "workspace", false));
    const Range writes[] = {{data, (size_t)M * K, "data"}, {scales, (size_t)M * 4, "scales"}, {workspace, workspace_bytes, "workspace"}};
    const Range reads[] = {{x, span(x_rows, ld, K, size), "x"}, {rows, (size_t)M * 4, "rows"}};
    BN_TRY(check_overlaps(writes, 3, reads, 2));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    Int8Args a = {};
    a.x = x;
    a.ld = ld;
    a.x_rows = x_rows;
    a.rows = rows;
    a.M = M;
    a.K = K;
    a.data = data;
    a.scales = scales;
    a.err = d->err;
    const size_t need = rows ? bn_quantize_int8_workspace_bytes(x_rows, M, K) : 0;
    if (need && workspace && workspace_bytes >= need) {  // the rows of x once, then to their places
        a.rows = nullptr;
        a.M = x_rows;
        a.data = static_cast<int8_t *>(workspace);
        a.scales = reinterpret_cast<float *>(a.data + (size_t)x_rows * K);
        BN_TRY(launched(launch_quantize_int8(a, dtype, dependent_launch(), (cudaStream_t)stream), "launching quantize_int8"));
        return launched(launch_place_rows(a.data, K / 2, x_rows, rows, M, nullptr, 0, K / 2, data, a.scales, scales, d->err, d->sms,
                                          dependent_launch(), (cudaStream_t)stream), "launching place_rows");
    }
    return launched(launch_quantize_int8(a, dtype, dependent_launch(), (cudaStream_t)stream), "launching quantize_int8");
}

bn_status bn_dequantize_int8(const int8_t *data, const float *scales, int M, int K, void *out, bn_dtype dtype,
                             void *stream)
{
    clear_message();
    BN_TRY(check_dtype(dtype, true));
    BN_TRY(check_int8(M, K));
    if (M == 0) return BN_OK;
    BN_TRY(check_ptr16(data, "data"));
    BN_TRY(check_ptr4(scales, "scales"));
    BN_TRY(check_ptr16(out, "out"));
    const Range writes[] = {{out, (size_t)M * K * dtype_size(dtype), "out"}};
    const Range reads[] = {{data, (size_t)M * K, "data"}, {scales, (size_t)M * 4, "scales"}};
    BN_TRY(check_overlaps(writes, 1, reads, 2));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    Int8Args a = {};
    a.M = M;
    a.K = K;
    a.data = const_cast<int8_t *>(data);
    a.scales = const_cast<float *>(scales);
    a.out = out;
    return launched(launch_dequantize_int8(a, dtype, dependent_launch(), (cudaStream_t)stream),
                    "launching dequantize_int8");
}

size_t bn_expert_product_int8_workspace_bytes(int M, int E, int N, int K)
{
    if (M < 1 || E < 1 || N < 8 || N % 8 != 0 || K < 16 || K % 16 != 0) return 0;
    Product8Args p = {};
    p.M = M;
    p.E = E;
    p.N = N;
    p.K = K;
    int split;
    return product8_pairs(p, kNominalSms, &split) ? (size_t)M * K * 2 : 0;
}

bn_status bn_expert_product_int8(const int8_t *a, const float *a_scales, int M, const int8_t *w, const float *w_scales,
                                 int E, int N, int K, const int32_t *offsets, float alpha, uint16_t *out,
                                 void *workspace, size_t workspace_bytes, void *stream)
{
    clear_message();
    BN_TRY(check_int8(M, K));
    BN_REQUIRE(E >= 1, "E=%d is not positive", E);
    BN_REQUIRE(N >= 8 && N % 8 == 0, "N=%d is not a positive multiple of 8", N);
    BN_REQUIRE(offsets || E == 1, "offsets is NULL with E=%d experts", E);
    BN_REQUIRE(aligned(offsets, 4), "offsets is not 4-byte aligned");
    BN_REQUIRE(std::isfinite(alpha), "alpha must be finite");
    if (E > kMaxExperts) return fail(BN_ERR_UNSUPPORTED, "E=%d above the served maximum %d", E, kMaxExperts);
    if (N > (1 << 20)) return fail(BN_ERR_UNSUPPORTED, "N=%d above the served maximum %d", N, 1 << 20);
    if (M == 0) return BN_OK;
    BN_TRY(check_ptr16(a, "a"));
    BN_TRY(check_ptr4(a_scales, "a_scales"));
    BN_TRY(check_ptr16(w, "w"));
    BN_TRY(check_ptr4(w_scales, "w_scales"));
    BN_TRY(check_ptr16(out, "out"));
    BN_TRY(check_ptr16(workspace, "workspace", false));
    const Range writes[] = {{out, (size_t)M * N * 2, "out"}, {workspace, workspace_bytes, "workspace"}};
    const Range reads[] = {{a, (size_t)M * K, "a"},
                           {a_scales, (size_t)M * 4, "a_scales"},
                           {w, (size_t)E * N * K, "w"},
                           {w_scales, (size_t)E * N * 4, "w_scales"},
                           {offsets, (size_t)(E + 1) * 4, "offsets"}};
    BN_TRY(check_overlaps(writes, 2, reads, 5));
    const DeviceInfo *d = nullptr;
    BN_TRY(device_info(&d));
    Product8Args p = {};
    p.M = M;
    p.E = E;
    p.N = N;
    p.K = K;
    p.offsets = offsets;
    p.a = a;
    p.a_scales = a_scales;
    p.w_scales = w_scales;
    p.alpha = alpha;
    p.out = out;
    p.err = d->err;
    void *wide = workspace_bytes >= (size_t)M * K * 2 ? workspace : nullptr;
    return launched(launch_product8(p, w, wide, d->sms, dependent_launch(), (cudaStream_t)stream),
                    "launching expert_product_int8");
}

}  // extern "C"
