// gdr_once.h -- a number asked once for each device and kept.  Plain C++.  Not
// part of the ABI.
#pragma once

#include <atomic>

namespace gdr {

class OncePerDevice {
public:
    // The number of device `dev`: what `ask` says (positive) the first time, else
    // `otherwise`, which is not kept.  Threads that ask at the same time keep the
    // same number.
    template <typename F>
    int get(int dev, int otherwise, F ask) {
        if (dev < 0 || dev >= kDevices) return otherwise;
        int n = known_[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
        n = ask();
        if (n <= 0) return otherwise;
        known_[dev].store(n, std::memory_order_relaxed);
        return n;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices] = {};
};

}  // namespace gdr
