// A number that is asked for once on each device.
#pragma once

#include <atomic>

namespace dflash {

class PerDevice {
 public:
  // What ask() gave for this device, the first time that it gave at least 1: a query that failed
  // is not kept.  (Devices past kMost are asked about every time.)
  template <typename Ask>
  int get(int device, Ask ask) {
    if (device < 0 || device >= kMost) return ask();
    int n = kept_[device].load(std::memory_order_relaxed);
    if (n < 1) {
      n = ask();
      if (n >= 1) kept_[device].store(n, std::memory_order_relaxed);
    }
    return n;
  }

 private:
  static constexpr int kMost = 64;
  std::atomic<int> kept_[kMost] = {};
};

}  // namespace dflash
