// What a launcher finds out once per device of the process: that a kernel's shared
// memory limit is raised (the limit belongs to the device's image of the kernel), how
// many of its clusters are resident, how many SMs there are.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace engram {

// A positive number per device, made on the current device at the first use there
// (by several threads at once, perhaps: each makes the same) and kept; 0 is not kept.
class PerDevice {
  public:
    // make(int*) -> cudaError_t; an error is returned, and the next use makes again.
    template <class Make>
    cudaError_t get(int* out, Make make) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool kept = dev >= 0 && dev < kDevices;
        int v = kept ? value_[dev].load(std::memory_order_acquire) : 0;
        if (v == 0) {
            e = make(&v);
            if (e != cudaSuccess) return e;
            if (kept) value_[dev].store(v, std::memory_order_release);
        }
        *out = v;
        return cudaSuccess;
    }

  private:
    static constexpr int kDevices = 64;  // (a device beyond these makes at every use)
    std::atomic<int> value_[kDevices] = {};
};

// Lets `kernel` be launched with up to `bytes` of dynamic shared memory on the current
// device: the same `bytes` at every call, so that no thread lowers another's limit.
template <class Kernel>
cudaError_t allow_shared(PerDevice& done, Kernel kernel, int bytes) {
    int v;
    return done.get(&v, [&](int* one) {
        *one = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
}

}  // namespace engram
