// What a launch sets up once per context of a device (again after a reset) and keeps.
#pragma once

#include <atomic>

#include "kernels.cuh"

namespace moe {

// Host threads may come for it at the same time.  The value is stored before the context that
// it holds for (release), and read after that context has been seen (acquire): who finds its
// own context here finds the value too.  Threads that both find nothing both set it up, to the
// same value.  Objects of this type are static (all zero: no context).
class OncePerContext {
 public:
  bool ready(int dev, unsigned long long ctx) const {
    return ctx != 0 && ctx_[dev].load(std::memory_order_acquire) == ctx;
  }
  int value(int dev) const { return value_[dev].load(std::memory_order_relaxed); }
  void set(int dev, int value) {
    value_[dev].store(value, std::memory_order_relaxed);
    ctx_[dev].store(current_context_id(), std::memory_order_release);
  }
  static constexpr int kDevices = 64;

 private:
  std::atomic<unsigned long long> ctx_[kDevices] = {};
  std::atomic<int> value_[kDevices] = {};
};

}  // namespace moe
