// SmemLimits over growing sizes, more kernels and devices than entries, refused sizes and two threads.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <thread>
#include <utility>

#include "smem_limits.h"

using Limits = std::map<std::pair<const void *, int>, int>;
static Limits limits;  // what the fake runtime holds; guarded by the table's own lock
static int calls = 0;

template <class T>
static bool raise(T &table, const void *kern, int dev, int bytes, int most = 1 << 30) {
    int &now = limits[{kern, dev}];
    return table.raise(
        kern, dev, bytes,
        [&](int b) {
            ++calls;
            if (b > most) return false;
            if (b < now) {
                std::printf("lowered from %d to %d\n", now, b);
                std::exit(1);
            }
            now = b;
            return true;
        },
        [&] { return now; });
}
static void check(bool ok, const char *what) {
    if (ok) return;
    std::printf("failed: %s\n", what);
    std::exit(1);
}
static const void *kernel(int i) { return reinterpret_cast<const void *>((uintptr_t)(0x4000 + 64 * i)); }

int main() {
    static w4a16::SmemLimits<> table;
    for (int b = 1000; b < 5000; ++b) check(raise(table, kernel(0), 0, b), "growing");
    check(calls == 4000, "a call for each larger size");
    for (int b = 1000; b < 5000; ++b) check(raise(table, kernel(0), 0, b), "smaller");
    check(calls == 4000, "none for smaller ones");
    // More kernels after one that took many sizes, on sixteen devices.
    for (int round = 0; round < 3; ++round)
        for (int dev = 0; dev < 16; ++dev)
            for (int k = 1; k <= 110; ++k) check(raise(table, kernel(k), dev, 100000 - 1000 * round), "many");
    check(calls == 4000 + 16 * 110, "one call each");
    check(!raise(table, kernel(500), 0, 300000, 232448) && raise(table, kernel(500), 0, 200000, 232448), "refused, then taken");

    static w4a16::SmemLimits<64> small;
    limits.clear();
    for (int round = 0; round < 3; ++round)
        for (int dev = 0; dev < 2; ++dev)
            for (int k = 0; k < 60; ++k) {
                check(raise(small, kernel(k), dev, round == 1 ? 60000 : 100000), "full table");
                check(limits[{kernel(k), dev}] >= 100000, "kept");
            }
    calls = 0;
    for (int k = 0; k < 60; ++k) raise(small, kernel(k), 1, 100000);
    check(calls == 0, "no call for a size that a full table's kernel has");

    // Two threads, a large and a small size of the same kernel: at a launch the limit is large enough.
    static w4a16::SmemLimits<2> two;
    static int now = 0;
    const auto worker = [](int bytes) {
        for (int i = 0; i < 20000; ++i)
            two.raise(kernel(i % 5), 0, bytes, [&](int b) { return b >= now ? (now = b, true) : (std::exit(1), false); }, [] { return now; });
    };
    std::thread a(worker, 100000), b(worker, 50000);
    a.join();
    b.join();
    std::printf("ok\n");
    return 0;
}
