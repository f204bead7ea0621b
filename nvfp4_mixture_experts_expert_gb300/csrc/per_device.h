// What a kernel's launches need to know of a device (function attributes set,
// clusters that fit), worked out once for each.  Host code only.
#pragma once
#include <atomic>
#include <mutex>

namespace nvfp4 {

constexpr int kMaxDevices = 64;

// Status: a type whose value-initialised value means success (cudaError_t).
template <typename T, typename Status>
class PerDevice {
 public:
  // Points `out` at device `dev`'s value (0 <= dev < kMaxDevices), which the first
  // caller fills in by fill(T&) while the others wait.  A failed fill's status is
  // returned, and the next caller tries again.
  template <typename Fill>
  Status get(int dev, const T** out, Fill fill) {
    Slot& s = slots_[dev];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mutex_);
      if (!s.ready.load(std::memory_order_relaxed)) {
        const Status e = fill(s.value);
        if (e != Status{}) return e;
        s.ready.store(true, std::memory_order_release);
      }
    }
    *out = &s.value;
    return Status{};
  }

 private:
  struct Slot {
    std::atomic<bool> ready{false};
    T value{};
  };
  std::mutex mutex_;
  Slot slots_[kMaxDevices];
};

}  // namespace nvfp4
