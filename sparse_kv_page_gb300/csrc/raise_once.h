// raise_once.h - a setting that only ever goes up, one per device (host code).
#pragma once

#include <atomic>
#include <mutex>

namespace locks {

// Remembers the largest value that was set on each device and sets larger ones. `set` (returning
// 0 on success) runs under a lock: of two threads that both find their value too large, the one
// with the smaller value must not set it over the other's.
class RaiseOnce {
public:
    static constexpr int kDevices = 64;

    template <class Set>
    auto raise(int device, int value, Set set) -> decltype(set()) {
        std::atomic<int>& done = done_[device];
        if (done.load(std::memory_order_acquire) > value) return {};
        std::lock_guard<std::mutex> lock(mu_);
        if (done.load(std::memory_order_relaxed) > value) return {};
        const auto e = set();
        if (e == decltype(set()){}) done.store(value + 1, std::memory_order_release);
        return e;
    }

private:
    std::atomic<int> done_[kDevices] = {};       // 1 + the largest value set; 0: none
    std::mutex mu_;
};

}  // namespace locks
