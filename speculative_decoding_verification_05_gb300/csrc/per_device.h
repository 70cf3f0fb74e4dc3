// Settings of a kernel that a process makes once a device.
#pragma once

#include <atomic>
#include <mutex>

namespace sv {

// run(key, dev, set) calls set() once for a key and device and remembers it if
// it returned 0; nobody gets 0 before that call has ended. What set() does must
// be a function of the key alone. Entries are written once, under the lock;
// readers find them without it.
class OncePerDevice {
    static constexpr int kMost = 256;  // (with all taken, set() is called every time)
    struct Entry {
        std::atomic<const void*> key{nullptr};
        int dev = 0;
    };
    Entry seen_[kMost];
    std::mutex mu_;

    bool done(const void* key, int dev) const {
        for (const Entry& e : seen_) {
            const void* k = e.key.load(std::memory_order_acquire);
            if (!k) return false;
            if (k == key && e.dev == dev) return true;
        }
        return false;
    }

public:
    template <typename Set>
    int run(const void* key, int dev, Set set) {
        if (done(key, dev)) return 0;
        std::lock_guard<std::mutex> g(mu_);
        if (done(key, dev)) return 0;
        const int rc = set();
        if (rc != 0) return rc;
        for (Entry& e : seen_)
            if (!e.key.load(std::memory_order_relaxed)) {
                e.dev = dev;
                e.key.store(key, std::memory_order_release);
                break;
            }
        return 0;
    }
};

}  // namespace sv
