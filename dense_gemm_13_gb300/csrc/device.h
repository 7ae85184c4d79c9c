// device.h -- the current device, for calls without a plan; a plan's memory, when it goes.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace g13 {

// Whether the current device is an sm_103, and its SMs (asked once per device: an attribute costs
// a call of a few microseconds more on the host).
inline bool usable_device(int* sms, int* device = nullptr) {
    constexpr int kMost = 64;
    static std::atomic<int> known[kMost];  // SMs + 1; -1: not an sm_103
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
    if (device) *device = dev;
    int n = dev < kMost ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int major = 0, minor = 0, count = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return false;
        n = major == 10 && minor == 3 ? count + 1 : -1;
        if (dev < kMost) known[dev].store(n, std::memory_order_relaxed);
    }
    if (n < 0) return false;
    *sms = n - 1;
    return true;
}

// Frees a plan's memory.  A plan may be destroyed while this thread captures a graph (in Python, whenever the garbage
// collector finds it), where a plain cudaFree would spoil the capture.
inline void free_plan_memory(void* p) {
    if (!p) return;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool changed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    cudaFree(p);
    if (changed) cudaThreadExchangeStreamCaptureMode(&mode);
}

}  // namespace g13
