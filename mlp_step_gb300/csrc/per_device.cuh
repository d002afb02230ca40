// What a launcher finds out once per device: occupancy, and whether a kernel's
// limits are set (both belong to a device, not to the process).  Host code.
#pragma once

#include <atomic>

namespace mlp {

// A positive number per device, made on first use.  Threads that meet there
// make the same number; one that is not positive (a failure) is made again on
// the next call.
class PerDevice {
 public:
  template <typename F>
  int get(int device, F&& make) {
    if (device < 0 || device >= kDevices) return make();
    std::atomic<int>& v = value_[device];
    int n = v.load(std::memory_order_acquire);
    if (n > 0) return n;
    n = make();
    if (n > 0) v.store(n, std::memory_order_release);
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> value_[kDevices] = {};
};

}  // namespace mlp
