// per_device.h -- a number that the host finds out once for each device of the process.
#pragma once
#include <atomic>

namespace k3moe {

// A number >= 0 per device, zero-initialised where it is static.  Any threads may ask at the same time:
// two that come first may both find it out, and get the same.
class PerDevice {
 public:
  static constexpr int kDevices = 64;
  // The number of device `dev`: find()'s, from the first call on.  A negative one is a failure, and is not kept.
  template <class F>
  int get(int dev, F find) {
    const bool keep = dev >= 0 && dev < kDevices;
    const int known = keep ? known_[dev].load(std::memory_order_acquire) : 0;
    if (known) return known - 1;
    const int n = find();
    if (keep && n >= 0) known_[dev].store(n + 1, std::memory_order_release);
    return n;
  }

 private:
  std::atomic<int> known_[kDevices] = {};  // + 1; 0: not yet known
};

}  // namespace k3moe
