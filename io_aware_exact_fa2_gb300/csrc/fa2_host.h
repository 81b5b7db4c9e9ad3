// fa2_host.h -- what the host sides of both libraries (fa2_api.cu, fa2_cache_api.cu) share: a device's
// SM count, and limits of the kernels' bounded waits from the environment.
#pragma once

#include <cstdlib>
#include <mutex>

#include <cuda_runtime.h>

namespace fa2 {

constexpr int kMaxDevices = 64;

// Number of SMs of a device (looked up once per device); 0 if it cannot be told.
inline int sm_count(int dev)
{
    static std::mutex mu;
    static int cache[kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < kMaxDevices && cache[dev] > 0)
        return cache[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < kMaxDevices)
        cache[dev] = n;
    return n;
}

// Limit of the kernels' waits: one second, or FA2_WAIT_LIMIT_MS (read once).
inline unsigned long long wait_limit_ns()
{
    static const unsigned long long limit = [] {
        const char *s = std::getenv("FA2_WAIT_LIMIT_MS");
        const long long ms = s ? std::atoll(s) : 0;
        return static_cast<unsigned long long>(ms > 0 ? ms : 1000) * 1000000ull;
    }();
    return limit;
}

// Limit of a call's waits between warps.  FA2_TEST_WAIT_LIMIT_NS (read on every call, nanoseconds)
// shortens it so that a test of the time-out path ends quickly; the waits with which a CTA drains
// its own copies and MMAs before exiting keep the full limit.
inline unsigned long long call_wait_limit_ns()
{
    const char *s = std::getenv("FA2_TEST_WAIT_LIMIT_NS");
    const long long ns = s ? std::atoll(s) : 0;
    return ns > 0 ? static_cast<unsigned long long>(ns) : wait_limit_ns();
}

}  // namespace fa2
