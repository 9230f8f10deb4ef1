// host.hpp -- host-side pieces shared by the library's source files: the HIP
// error of the calling thread, the device check, and the argument checks
// (alignment, byte extents, overlap, caller workspaces).
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>
#include <mutex>
#include <stdint.h>
#include <string.h>

#include "dg_fp8.h"

namespace dgh {

inline thread_local int g_last_hip_error = 0;

struct DeviceInfo {
    bool known = false;
    bool gfx950 = false;
    int cus = 0;
};

constexpr int kMaxDevices = 64;
inline DeviceInfo g_devices[kMaxDevices];
inline std::mutex g_devices_mu;

inline int fail_hip(hipError_t e)
{
    g_last_hip_error = (int)e;
    return DG_ERR_HIP;
}

// Checks that the current device is gfx950 and caches its CU count.
inline int current_device(DeviceInfo &out)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return fail_hip(e);
    if (dev < 0 || dev >= kMaxDevices)
        return DG_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_devices_mu);
    DeviceInfo &d = g_devices[dev];
    if (!d.known) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess)
            return fail_hip(e);
        d.gfx950 = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
        d.cus = prop.multiProcessorCount;
        d.known = true;
    }
    out = d;
    return d.gfx950 ? DG_OK : DG_ERR_UNSUPPORTED;
}

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// [lo, hi) byte extent of a strided 2-D/3-D operand (all strides >= 0).
struct Extent {
    uintptr_t lo, hi;
};

inline Extent extent(const void *p, int64_t elem, int64_t last_index)
{
    const uintptr_t lo = (uintptr_t)p;
    return Extent{lo, lo + (uintptr_t)((last_index + 1) * elem)};
}

inline bool overlaps(Extent a, Extent b) { return a.lo < b.hi && b.lo < a.hi; }

constexpr int64_t kInt32Max = 0x7fffffff;

// A caller workspace must be 16-byte aligned, have a non-negative size and
// lie apart from the call's output and inputs.
inline int check_workspace(const void *ws, int64_t ws_bytes, std::initializer_list<Extent> others)
{
    if (ws_bytes < 0)
        return DG_ERR_BAD_SHAPE;
    if (!ws || ws_bytes == 0)
        return DG_OK;
    if (!aligned(ws, 16))
        return DG_ERR_MISALIGNED;
    const Extent ew = extent(ws, 1, ws_bytes - 1);
    for (const Extent &e : others)
        if (e.hi > e.lo && overlaps(ew, e))
            return DG_ERR_ALIASING;
    return DG_OK;
}

}  // namespace dgh
