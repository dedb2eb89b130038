// What the host remembers of a device: its SMs, and the shared memory that each
// kernel may use there.  Both belong to one device of the process: another one is
// asked, or told, for itself.  And how plans give back device memory.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace sga {

constexpr int kMaxDevices = 64;   // (past these nothing is remembered)

// The current device, -1 where nothing is remembered of it.
inline int remembered_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}

// A number of the current device, `look_up`'s (positive; 0: failed, and asked again) the first time.
template <typename F> int per_device(std::atomic<int> (&known)[kMaxDevices], F look_up) {
    const int dev = remembered_device();
    int n = dev < 0 ? 0 : known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    n = look_up();
    if (dev >= 0) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// SMs of the current device.
inline int device_sms() {
    static std::atomic<int> known[kMaxDevices];
    const int n = per_device(known, [] {
        int dev = 0, sms = 0;
        cudaGetDevice(&dev);
        return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? sms : 0;
    });
    return n < 1 ? 1 : n;
}

// Let Kernel launch with `smem` bytes of dynamic shared memory on the current
// device: raises its limit there whenever a launch needs more than any before it
// (kernels whose size depends on the call's shape would otherwise keep the first
// call's limit and refuse a larger launch).  Raised by one thread at a time: two
// at once could leave the smaller limit behind.
template <auto Kernel> cudaError_t allow_smem(size_t smem) {
    static std::atomic<size_t> allowed[kMaxDevices];
    static std::mutex raising;
    if (smem <= 48 * 1024) return cudaSuccess;   // (of every kernel)
    const int dev = remembered_device();
    if (dev >= 0 && smem <= allowed[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(raising);
    if (dev >= 0 && smem <= allowed[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && dev >= 0) allowed[dev].store(smem, std::memory_order_relaxed);
    return e;
}

// Frees a plan's memory.  A plan may be dropped at any time, also while some stream
// of the process is being captured (a collector may run then), and cudaFree would
// end that capture unless the thread says that it does not take part in it.
inline void free_device(void *p) {
    if (!p) return;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool set = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;   // (the mode before comes back in it)
    cudaFree(p);
    if (set) cudaThreadExchangeStreamCaptureMode(&mode);
}

}  // namespace sga
