// Host helpers shared by the C entry points of libbconv.so: the calling
// thread's error text, device selection, uploads and pointer checks.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "bconv.h"

namespace bconv {

// Text behind bconv_last_error().  A plain array, so that recording an error
// cannot itself fail or throw through a C entry point.
inline thread_local char last_error[512];

__attribute__((format(printf, 2, 3))) inline bconv_status_t fail(bconv_status_t s, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(last_error, sizeof last_error, fmt, ap);
    va_end(ap);
    return s;
}

inline bconv_status_t hip_fail(hipError_t e, const char *what)
{
    return fail(BCONV_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Runs `fn` with the handle's device current, restoring the caller's device.
struct DeviceGuard {
    int prev = -1;
    hipError_t err = hipSuccess;
    explicit DeviceGuard(int dev)
    {
        err = hipGetDevice(&prev);
        if (err == hipSuccess && prev != dev) err = hipSetDevice(dev);
        else if (err == hipSuccess) prev = -1;
    }
    ~DeviceGuard()
    {
        if (prev >= 0) (void)hipSetDevice(prev);
    }
};

template <typename T>
inline bconv_status_t upload(const T *host, size_t count, T **dev)
{
    *dev = nullptr;
    if (!host || count == 0) return BCONV_OK;
    hipError_t e = hipMalloc(reinterpret_cast<void **>(dev), count * sizeof(T));
    if (e != hipSuccess) {
        *dev = nullptr;
        return fail(BCONV_ERR_ALLOC, "hipMalloc(%zu): %s", count * sizeof(T), hipGetErrorString(e));
    }
    e = hipMemcpy(*dev, host, count * sizeof(T), hipMemcpyHostToDevice);
    if (e != hipSuccess) return hip_fail(e, "hipMemcpy");
    return BCONV_OK;
}

// Workgroups that one launch takes: the runtime counts a dimension's threads in
// 32 bits, and no workgroup here has more than 512 threads.
constexpr long long kMaxGroups = 1LL << 22;

// Calls launch(first, count) for `total` workgroups, as many launches as they
// take (one, but for extreme sizes); the first error ends it.
template <typename F> inline hipError_t launch_slices(long long total, F launch)
{
    for (long long first = 0; first < total; first += kMaxGroups) {
        launch(first, (unsigned)(total - first < kMaxGroups ? total - first : kMaxGroups));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

inline bool ranges_overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bn && b0 < a0 + an;
}

}  // namespace bconv
