// per_device.h -- host values that belong to one CUDA device: the address of a __device__ variable,
// whether a kernel's shared memory limit has been raised, the number of SMs.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace osm {

// A value made once for each device, by the first call with that device current.  make(device)
// returns T{} (0, false, nullptr) where it fails; a failure is not kept, and neither is the value of a
// device past the last slot.  Two first calls at once may both make it, so making it twice must do no
// harm.
template <typename T>
class PerDevice {
public:
    template <typename Make>
    T get(const Make& make) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return T{};
        if (dev < 0 || dev >= kSlots) return make(dev);
        T v = slots_[dev].load(std::memory_order_acquire);
        if (v == T{}) {
            v = make(dev);
            if (v != T{}) slots_[dev].store(v, std::memory_order_release);
        }
        return v;
    }

private:
    static constexpr int kSlots = 64;
    std::atomic<T> slots_[kSlots] = {};
};

// SMs of the current device; 0 when they cannot be had.
inline int device_sm_count() {
    static PerDevice<int> sms;
    return sms.get([](int dev) {
        int n = 0;
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? n : 0;
    });
}

}  // namespace osm
