// What the C entry points share: the thread's last error, and the checks of
// pointers, sizes, workspaces and the device.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/bsg.h"

namespace bsg {
namespace api {

inline thread_local char g_err[512] = "";

inline int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return status;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_bytes(int dt)
{
    switch (dt) {
    case BSG_F32: return 4;
    case BSG_F16:
    case BSG_BF16: return 2;
    default: return 1;
    }
}

inline bool is_float_out(int dt) { return dt == BSG_F32 || dt == BSG_F16 || dt == BSG_BF16; }

// Device check: the kernels are built for gfx950 only.
inline int check_device()
{
    static int cached[64];   // 0 unknown, 1 ok, 2 bad
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return fail(BSG_ERR_DEVICE, "hipGetDevice failed");
    if (dev >= 0 && dev < 64 && cached[dev] == 1) return BSG_OK;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return fail(BSG_ERR_DEVICE, "hipGetDeviceProperties failed");
    if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) {
        if (dev >= 0 && dev < 64) cached[dev] = 2;
        return fail(BSG_ERR_DEVICE, "device %d is %s; this library is built for gfx950", dev,
                    prop.gcnArchName);
    }
    if (dev >= 0 && dev < 64) cached[dev] = 1;
    return BSG_OK;
}

inline int launch_status(hipError_t e, const char *what)
{
    if (e == hipSuccess) return BSG_OK;
    if (e == hipErrorNotSupported) return fail(BSG_ERR_UNSUPPORTED, "%s: not supported", what);
    return fail(BSG_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
}

inline bool is_16bit(int dt) { return dt == BSG_F16 || dt == BSG_BF16; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// sizes of a product, or of tokens and channels
inline int check_ffn_sizes(int64_t m, int64_t n, int64_t k)
{
    if (m < 0 || n < 0 || k < 0) return fail(BSG_ERR_SHAPE, "negative size");
    if (m > (1ll << 22) || n > (1ll << 20) || k > (1ll << 20))
        return fail(BSG_ERR_UNSUPPORTED, "M=%lld, N=%lld, K=%lld: past 2^22 tokens or 2^20 channels", (long long)m,
                    (long long)n, (long long)k);
    return BSG_OK;
}

// output tiles of an (r, c) product: the grid's limit
inline int check_ffn_tiles(int64_t r, int64_t c)
{
    const int64_t tiles = ((r + 63) / 64) * ((c + 63) / 64);
    if (tiles >= (1ll << 23)) return fail(BSG_ERR_UNSUPPORTED, "%lld output tiles exceed the launch limit", (long long)tiles);
    return BSG_OK;
}

inline int check_workspace(const void *ws, int64_t have, int op, int64_t m, int64_t n, int64_t k)
{
    const int64_t need = bsg_workspace_bytes(op, m, n, k);
    if (need == 0) return BSG_OK;
    if (!ws) return fail(BSG_ERR_NULLPTR, "a workspace of %lld bytes is required", (long long)need);
    if (!aligned16(ws)) return fail(BSG_ERR_ALIGN, "workspace must be 16-byte aligned");
    if (have < need)
        return fail(BSG_ERR_SHAPE, "workspace holds %lld bytes; these sizes need %lld", (long long)have, (long long)need);
    return BSG_OK;
}

}  // namespace api
}  // namespace bsg
