// What has to be done once on every device that a process uses, such as raising a kernel's
// shared-memory limit (a kernel's attributes belong to a device).
#pragma once

#include <atomic>
#include <cstdint>

namespace pa {

class DeviceOnce {
public:
    // Calls set() unless it has succeeded on device `dev` before; false if it fails (it is
    // tried again by the next call) or dev is none of 0 .. 63.  Threads that call at once may
    // both call set().
    template <typename F>
    bool operator()(int dev, F set) {
        if (dev < 0 || dev >= 64) return false;
        if (done_.load(std::memory_order_acquire) >> dev & 1) return true;
        if (!set()) return false;
        done_.fetch_or(uint64_t(1) << dev, std::memory_order_release);
        return true;
    }

private:
    std::atomic<uint64_t> done_{0};
};

}  // namespace pa
