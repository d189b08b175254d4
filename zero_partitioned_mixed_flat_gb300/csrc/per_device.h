// per_device.h -- what a process finds out once about each device (host only).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace zk {

// A positive number for every device that calls run on: a kernel's occupancy, or that its
// shared memory has been allowed.  Both hold for the device that was current when
// they were asked for, and for no other.  What is not positive (a call that failed) is
// not kept.  Threads may ask at once: they find the same.
class PerDevice {
  public:
    static constexpr int kDevices = 64;

    template <typename Find>
    int get(Find &&find) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return -(int)e;
        if (dev < 0 || dev >= kDevices) return find();
        int n = kept_[dev].load(std::memory_order_acquire);
        if (n > 0) return n;
        n = find();
        if (n > 0) kept_[dev].store(n, std::memory_order_release);
        return n;
    }

  private:
    std::atomic<int> kept_[kDevices] = {};
};

// a call's status as such a number: 1, or the error below zero
inline int done_or_error(cudaError_t e) { return e == cudaSuccess ? 1 : -(int)e; }

}  // namespace zk
