// Positive counts that depend on the device, asked for once per device and slot.
#pragma once

#include <atomic>

namespace uno {

template <int kSlots>
class PerDevice {
 public:
  // The count of `slot` on `device`: kept from an earlier call, or ask() (devices
  // past the table are asked each time). Threads that meet here ask twice at most.
  template <typename Ask>
  int get(int device, int slot, const Ask& ask) {
    if (device < 0 || device >= kDevices || slot < 0 || slot >= kSlots) return ask();
    std::atomic<int>& kept = kept_[device][slot];
    if (const int n = kept.load(std::memory_order_relaxed)) return n;
    const int n = ask();
    kept.store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> kept_[kDevices][kSlots] = {};
};

}  // namespace uno
