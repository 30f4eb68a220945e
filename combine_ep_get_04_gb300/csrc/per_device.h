// per_device.h -- answers that a device gives once and that do not change, as
// plain host code, so that it is checked on the CPU against a fake device.
#pragma once

#include <atomic>

namespace ep {

constexpr int kKnownDevices = 64;

// Positive answers to KINDS questions, of each device.  Several threads may ask at once.
template <int KINDS>
class PerDevice {
  public:
    // What `device` has answered to question `kind`, or answers now: ask(&answer) is true where it did.  Where it does
    // not, `otherwise` serves this once.
    template <typename Ask>
    int get(int device, int kind, int otherwise, Ask ask) {
        std::atomic<int>* at = device >= 0 && device < kKnownDevices ? &known_[device][kind] : nullptr;
        int n = at != nullptr ? at->load(std::memory_order_relaxed) : 0;
        if (n > 0) return n;
        if (!ask(&n) || n < 1) return otherwise;
        if (at != nullptr) at->store(n, std::memory_order_relaxed);
        return n;
    }

  private:
    std::atomic<int> known_[kKnownDevices][KINDS] = {};          // 0: not asked yet
};

}  // namespace ep
