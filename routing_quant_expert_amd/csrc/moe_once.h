// What a launch has to set up once on every device (host code, no HIP types).
#pragma once

#include <atomic>
#include <cstdint>

namespace moe {

// set_up(), an error code whose 0 is success, for each device until it has
// succeeded there: a failure is returned, and tried again by the next call.
// (Threads that come at once may each set up: it does no harm twice.)
class OncePerDevice {
  std::atomic<uint64_t> done_{0};   // devices 0..63; others are set up by every call

 public:
  template <class F>
  auto operator()(int device, F&& set_up) -> decltype(set_up()) {
    typedef decltype(set_up()) Error;
    const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return (Error)0;
    const Error e = set_up();
    if (e == (Error)0) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

}  // namespace moe
