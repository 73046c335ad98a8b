// Host helper of the launches that need more than 48 KiB of shared memory.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace pa {

// The opt-in to `bytes` of dynamic shared memory for a kernel, once per device (raised): asked
// for at each launch it costs the host about 2 us.
constexpr int kRaisedDevices = 64;
inline cudaError_t raise_shared_memory(std::atomic<bool> (&raised)[kRaisedDevices],
                                       const void *kernel, int bytes)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kRaisedDevices)
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (raised[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        raised[dev].store(true, std::memory_order_release);
    return e;
}

} // namespace pa
