// pa_host.cuh -- host helpers of the cache operators: current device and its
// SM count, pointer alignment, launches that may start while the previous
// kernel in the stream still runs (programmatic dependent launch).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace pa {

constexpr int kHostDevices = 64;

inline bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// Current device and its SMs (cached per device); false if CUDA reports an error.
inline bool device_and_sms(int* dev, int* sms) {
    static std::atomic<int> cache[kHostDevices];
    if (cudaGetDevice(dev) != cudaSuccess || *dev < 0) return false;
    int v = *dev < kHostDevices ? cache[*dev].load() : 0;
    if (v <= 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) return false;
        if (*dev < kHostDevices) cache[*dev].store(v);
    }
    *sms = v;
    return true;
}

// The kernel waits for the previous one (griddepcontrol.wait) before it touches
// anything that one may read or write.
template <class P>
bool launch_pdl(void (*kernel)(P), dim3 grid, int threads, size_t smem, void* stream, const P& params) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params) == cudaSuccess;
}

}  // namespace pa
