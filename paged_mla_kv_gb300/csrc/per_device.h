// What the library works out once for each GPU of the process (opt-ins, SM and cluster counts).
#pragma once

#include <atomic>
#include <mutex>

namespace tf {

constexpr int kMaxDevices = 64;

// One T a device.  get(dev, make) has make(T &) fill it in, which returns whether it could; a failure is
// not kept, so the next call asks again.  Null for a device past the table and after a failure.
template <typename T>
class PerDevice {
    std::mutex mu;
    std::atomic<bool> ready[kMaxDevices] = {};
    T value[kMaxDevices] = {};

   public:
    template <typename F>
    const T *get(int dev, F &&make) {
        if (dev < 0 || dev >= kMaxDevices) return nullptr;
        if (ready[dev].load(std::memory_order_acquire)) return &value[dev];
        std::lock_guard<std::mutex> g(mu);
        if (!ready[dev].load(std::memory_order_relaxed)) {
            T t = {};
            if (!make(t)) return nullptr;
            value[dev] = t;
            ready[dev].store(true, std::memory_order_release);
        }
        return &value[dev];
    }
};

}  // namespace tf
