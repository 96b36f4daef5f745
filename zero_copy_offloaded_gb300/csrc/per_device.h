// A setting that a process makes once for each device, whichever host thread comes first.
#pragma once

#include <atomic>

namespace dkv {

struct PerDevice {
  std::atomic<bool> done[64] = {};

  // `set` returns 0 for success.  Threads that come at once may both call it, so it must be one that
  // can be repeated; behind the 64th device it is called each time.
  template <typename F>
  auto operator()(int device, F&& set) -> decltype(set()) {
    const bool kept = device >= 0 && device < 64;
    if (kept && done[device].load(std::memory_order_acquire)) return {};
    const auto e = set();
    if (kept && !static_cast<int>(e)) done[device].store(true, std::memory_order_release);
    return e;
  }
};

}  // namespace dkv
