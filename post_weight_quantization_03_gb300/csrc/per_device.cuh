// Host-side numbers that belong to a device and are asked for once (plain C++).
#pragma once

#include <atomic>

namespace gptq {

// Positive numbers by device and key.
template <int KEYS>
class PerDevice {
 public:
  // The number of (dev, key): query() the first time and as long as it fails (gives less than 1),
  // which is answered with `otherwise` and not kept.
  template <typename Query>
  int get(int dev, int key, Query query, int otherwise) {
    const bool kept = dev >= 0 && dev < kDevices && key >= 0 && key < KEYS;
    int n = kept ? known_[dev][key].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    n = query();
    if (n < 1) return otherwise;
    if (kept) known_[dev][key].store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  static constexpr int kDevices = 128;
  std::atomic<int> known_[kDevices][KEYS] = {};
};

}  // namespace gptq
