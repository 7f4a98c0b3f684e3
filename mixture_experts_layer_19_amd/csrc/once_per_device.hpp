// once_per_device.hpp -- a setting that belongs to a kernel on one device (internal;
// plain C++).
#pragma once
#include <atomic>
#include <stdint.h>

namespace moe {

// set() for each device until it returned 0 there; its result, or 0 where it was
// set before.  A failure is not kept.  Devices past 63 are set at every call.
class OncePerDevice {
  std::atomic<uint64_t> done{0};

 public:
  template <typename Set>
  int operator()(int device, Set &&set) {
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return 0;
    const int err = set();
    if (err == 0) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
  }
};

}  // namespace moe
