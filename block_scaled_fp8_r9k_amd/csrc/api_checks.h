// Argument checks shared by the C ABI files of the 4-bit and 8-bit weights, the rows
// sorted by expert and the router.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>
#include <initializer_list>

#include "r9k.h"

namespace r9k {

// Device check, cached per device id: 1 = gfx950, 2 = not usable.
inline constexpr int MAX_DEV = 64;
inline std::atomic<int> g_dev_ok[MAX_DEV];

inline int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return R9K_ERR_DEVICE;
    }
    const int st = dev < MAX_DEV ? g_dev_ok[dev].load() : 0;
    if (st) return st == 1 ? R9K_OK : R9K_ERR_DEVICE;
    hipDeviceProp_t prop;
    const bool ok = hipGetDeviceProperties(&prop, dev) == hipSuccess && strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    (void)hipGetLastError();
    if (dev < MAX_DEV) g_dev_ok[dev] = ok ? 1 : 2;
    return ok ? R9K_OK : R9K_ERR_DEVICE;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline int launch_result(hipError_t e) { return e == hipSuccess ? R9K_OK : R9K_ERR_LAUNCH; }

inline constexpr int64_t MAX_DIM = int64_t(1) << 24;

// Blocks of 256 threads in a launch: the runtime refuses 2^32 threads and more
inline constexpr int64_t MAX_BLOCKS = int64_t(1) << 24;

// Experts that the sort and the expert products take: the sort keeps four counters an
// expert in a CTA's LDS
inline constexpr int64_t MOE_MAX_E = 2048;

// Bytes that a call reads or writes.  Its CTAs read while others write, so an output
// (a workspace too) may lie on no input and on no other output.
struct Span {
    const void *p;
    int64_t n;
};
inline bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.n > 0 && b.n > 0 && x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n;
}
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(*o, i)) return true;
        for (auto q = outs.begin(); q != o; ++q)
            if (overlap(*o, *q)) return true;
    }
    return false;
}

}  // namespace r9k
