// The dynamic shared-memory limits that kernels have been given: host code alone.
#pragma once

#include <atomic>
#include <cstddef>
#include <mutex>

namespace lora {

// Per kernel and device the largest size a launch has asked for.  A limit is set by
// an assignment to the kernel, so two threads that raise the same one must not pass
// each other: the smaller would be the last to be set and stay below what the table
// says.  Raising is therefore done under a lock; a size within the limit takes none.
template <int kSlots, int kDevices>
class SmemLimits {
 public:
  // set(): gives the kernel the limit `bytes` on the device, 0 if that worked.
  // Returns what set() did, 0 without a call where the limit is there already.
  template <typename Set>
  int raise(const void* func, int dev, size_t bytes, Set set) {
    const int slot = find(func);
    if (slot >= 0 && limit_[slot][dev].load(std::memory_order_acquire) >= bytes) return 0;
    std::lock_guard<std::mutex> lock(mu_);
    if (slot >= 0 && limit_[slot][dev].load(std::memory_order_relaxed) >= bytes) return 0;
    const int e = set();
    if (e == 0 && slot >= 0) limit_[slot][dev].store(bytes, std::memory_order_release);
    return e;
  }

 private:
  // The kernel's slot, its own from the first call on; -1 when the table is full.
  int find(const void* func) {
    for (int i = 0; i < kSlots; ++i) {
      const void* f = funcs_[i].load();
      if (f == func) return i;
      if (f == nullptr) {
        const void* expected = nullptr;
        if (funcs_[i].compare_exchange_strong(expected, func) || expected == func) return i;
      }
    }
    return -1;
  }

  std::mutex mu_;
  std::atomic<size_t> limit_[kSlots][kDevices] = {};
  std::atomic<const void*> funcs_[kSlots] = {};
};

}  // namespace lora
