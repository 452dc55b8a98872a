// per_device.h - what has to be done once on each device that a process uses, by whichever thread comes first.
#pragma once

#include <atomic>

namespace uw {

class OncePerDevice {
    static constexpr int kDevices = 64;  // beyond, every time
    std::atomic<bool> done_[kDevices] = {};

public:
    // f() until it has returned 0 for this device; returns what it did.  Threads at once may each run it.
    template <typename F>
    int operator()(int device, F f)
    {
        const bool kept = device >= 0 && device < kDevices;
        if (kept && done_[device].load(std::memory_order_acquire)) return 0;
        const int e = f();
        if (kept && e == 0) done_[device].store(true, std::memory_order_release);
        return e;
    }
};

}  // namespace uw
