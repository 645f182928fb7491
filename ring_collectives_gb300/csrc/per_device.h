// per_device.h -- settings that CUDA keeps per device, such as a kernel's
// limit on dynamic shared memory (host code only).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace rc {

class OncePerDevice {
public:
    // Runs `set` unless it already succeeded on the current device.  What it
    // returns is returned, and after a failure the next call tries again.  Two
    // threads may run it at once, so it has to bear repeating.
    template <class F>
    cudaError_t operator()(F set)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = set();
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> done{0};
};

} // namespace rc
