// per_device.h — what a process sets once for each GPU it uses. Plain C++ without HIP's headers, so
// that the tests run it on the CPU.
#pragma once
#include <atomic>
#include <cstdint>

namespace coli {

// set() on the first call of each device; a set that fails is tried again by the next call. Calls
// that race may both set: set() has to bear that. Devices past 63 are set every time.
struct PerDevice {
  std::atomic<uint64_t> done{0};

  template <typename Set>
  auto once(int device, Set set) -> decltype(set()) {
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_acquire) & bit) return decltype(set())(0);
    const auto st = set();
    if (st == decltype(set())(0)) done.fetch_or(bit, std::memory_order_release);
    return st;
  }
};

}  // namespace coli
