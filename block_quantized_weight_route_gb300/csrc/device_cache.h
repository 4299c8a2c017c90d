// What the launchers ask the CUDA runtime once per device.
#pragma once
#include <atomic>

namespace qmm {

constexpr int kMaxDevices = 64;

// One positive int per device, 0 until it is known.  The library may be called from
// several threads: two that find 0 at once both ask, and store the same.
class PerDevice {
public:
    int get(int dev) const { return v_[dev].load(std::memory_order_acquire); }
    void set(int dev, int value) { v_[dev].store(value, std::memory_order_release); }

private:
    std::atomic<int> v_[kMaxDevices] = {};
};

}  // namespace qmm
