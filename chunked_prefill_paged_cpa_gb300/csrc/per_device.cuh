// A number that belongs to a device and is found out, or set up, on first use
// there: the attributes of a kernel that have been set, the CTAs that an SM
// holds.  A process may use several devices, from several threads.
// (Plain C++: no CUDA header is needed to compile this one.)
#pragma once

#include <atomic>

namespace cpa {

class PerDevice {
 public:
  // The device's number, which is positive.  Where it has none yet, make() gives
  // it; what make() returns below 1 (a failure) is returned and not kept.
  // (Threads that come at once may each make it.)
  template <class Make>
  int get(int device, Make make) {
    if (device < 0 || device >= kDevices) return make();
    int x = known_[device].load(std::memory_order_acquire);
    if (x < 1) {
      x = make();
      if (x > 0) known_[device].store(x, std::memory_order_release);
    }
    return x;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> known_[kDevices] = {};
};

}  // namespace cpa
