// once.cuh -- host work that is done once on each device.
#pragma once

#include <atomic>

#include <cuda_runtime_api.h>
#include <stdint.h>

namespace dsa {

// A kernel's attributes, set once on each device that launches it (they belong
// to the device's own copy of the kernel, and setting them takes longer than
// the rest of a launch's preparation).
struct OncePerDevice {
    std::atomic<uint64_t> done{0};
    template <typename F>
    cudaError_t run(F set) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
        if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        const cudaError_t r = set();
        if (r == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return r;
    }
};

}  // namespace dsa
