// Host only: answers of the runtime that results depend on, asked for once a device.
#pragma once
#include <atomic>

namespace e0 {

// The first answer to each of N questions on each device, and no other afterwards.  Without
// an answer (ask gives less than 1) `otherwise` counts from then on; a device beyond the
// table is never asked.
template <int N>
class FirstAnswer {
public:
    template <typename F>
    int get(int dev, int which, int otherwise, F ask) {
        if (dev < 0 || dev >= DEVICES) return otherwise;
        std::atomic<int>& known = known_[dev][which];
        int n = known.load(std::memory_order_relaxed);
        if (n > 0) return n;
        int now = ask();
        if (now < 1) now = otherwise;
        return known.compare_exchange_strong(n, now, std::memory_order_relaxed) ? now : n;
    }

private:
    static constexpr int DEVICES = 64;
    std::atomic<int> known_[DEVICES][N] = {};
};

}  // namespace e0
