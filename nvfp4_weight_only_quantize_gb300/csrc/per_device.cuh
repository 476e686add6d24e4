// Set-up that the process does once on each of its devices (host code only).
#pragma once

#include <atomic>

namespace qerl {

constexpr int kMaxDevices = 64;

// Runs `set` (0 when it is done) the first time that device `dev` asks; what fails is returned and tried again the next
// time.  `set` may run twice where two threads ask at once.
class OncePerDevice {
    std::atomic<bool> done_[kMaxDevices] = {};

  public:
    template <class F>
    auto operator()(int dev, F set) -> decltype(set())
    {
        using Status = decltype(set());
        if (dev >= 0 && dev < kMaxDevices && done_[dev].load(std::memory_order_acquire)) return Status(0);
        const Status st = set();
        if (st == Status(0) && dev >= 0 && dev < kMaxDevices) done_[dev].store(true, std::memory_order_release);
        return st;
    }
};

}  // namespace qerl
