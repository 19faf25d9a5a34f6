// The dynamic shared-memory limits of kernels that this process has raised, by
// kernel and device: a limit is raised where a launch needs more than it, and
// never lowered, so that a launch captured into a graph makes no attribute call
// once its size was seen, and two host threads cannot take a limit from each
// other between its setting and the launch.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace w4a16 {

// kEntries: some hundred kernels on each of 16 devices, half full.  Past that a
// kernel's present limit is asked for, at every launch.
template <int kEntries = 4096>
class SmemLimits {
    struct Entry {
        const void *kern;  // null: free
        int dev, bytes;
    };
    std::mutex mu_;
    Entry entries_[kEntries] = {};

    // The kernel's entry, or a free one; null where neither is there.
    Entry *find(const void *kern, int dev) {
        const uint64_t h = (uint64_t)reinterpret_cast<uintptr_t>(kern) * 0x9E3779B97F4A7C15ull + (uint64_t)dev * 0xD6E8FEB86659FD93ull;
        unsigned at = (unsigned)(h >> 32) % kEntries;
        for (int i = 0; i < kEntries; ++i, at = (at + 1) % kEntries) {
            Entry &e = entries_[at];
            if (!e.kern || (e.kern == kern && e.dev == dev)) return &e;
        }
        return nullptr;
    }

   public:
    // Makes the limit at least `bytes`.  set(bytes) sets it, get() gives the present
    // one; false where set fails.
    template <class Set, class Get>
    bool raise(const void *kern, int dev, int bytes, Set set, Get get) {
        std::lock_guard<std::mutex> lock(mu_);
        Entry *e = find(kern, dev);
        if (e ? e->kern && e->bytes >= bytes : get() >= bytes) return true;
        if (!set(bytes)) return false;
        if (e) *e = Entry{kern, dev, bytes};
        return true;
    }
};

}  // namespace w4a16
