// bn_host.h -- host-side helpers shared by the C-ABI translation units: the
// error message, per-device facts, and argument checks (not part of the ABI).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/beamnorm.h"

namespace bn {

// Record the calling thread's message and return `st`.
bn_status fail(bn_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
bn_status cuda_fail(cudaError_t e, const char *what);
void clear_message();

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;      // dynamic + static shared memory one CTA may use
    int smem_per_sm = 0;     // shared memory of one SM
    int smem_reserved = 0;   // shared memory the system reserves per CTA
    unsigned *err = nullptr;  // address of g_bn_device_error on this device
};

// Facts of the current device, looked up once per device.
bn_status device_info(const DeviceInfo **out);

// A buffer of the call, for the overlap checks.
struct Range {
    const void *p;
    size_t bytes;
    const char *name;
};

bool aligned(const void *p, size_t a);
bn_status check_overlaps(const Range *writes, int nw, const Range *reads, int nr);
bn_status check_ptr16(const void *p, const char *name, bool required = true);
bn_status check_ptr4(const void *p, const char *name);

// 1 if launches carry programmatic dependent launch (bn_tuning.dependent_launch).
bool dependent_launch();

}  // namespace bn

#define BN_REQUIRE(cond, ...)                                            \
    do {                                                                 \
        if (!(cond)) return ::bn::fail(BN_ERR_INVALID, __VA_ARGS__);     \
    } while (0)
#define BN_TRY(expr)                         \
    do {                                     \
        bn_status _st = (expr);              \
        if (_st != BN_OK) return _st;        \
    } while (0)
