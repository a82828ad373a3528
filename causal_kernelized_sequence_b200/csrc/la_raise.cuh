// la_raise.cuh -- a limit that host threads raise, never lower (host code only).
#pragma once

#include <atomic>
#include <cstddef>
#include <mutex>

namespace la {

// to(want, set): calls set(want) unless the limit is known to be at least `want`
// already; what set returns false for is not remembered.  Check, call and note
// are one step: with two threads between them, a smaller limit could be set last
// and the larger one be remembered.  A limit that is high enough takes one load.
class Raise {
    std::atomic<size_t> done_{0};
    std::mutex one_;

public:
    template <typename F>
    bool to(size_t want, F set)
    {
        if (done_.load(std::memory_order_acquire) >= want) return true;
        std::lock_guard<std::mutex> hold(one_);
        if (done_.load(std::memory_order_relaxed) >= want) return true;
        if (!set(want)) return false;
        done_.store(want, std::memory_order_release);
        return true;
    }
};

}  // namespace la
