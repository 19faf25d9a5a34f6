// The rule by which the CTAs that share an item count their parts in and agree
// on who joins it: functions of the counts alone, which the kernels use and a
// host compiler can run over every order of counting.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define W4_RULE __device__ __forceinline__
#else
#define W4_RULE inline
#endif

namespace w4a16 {

// An item's count: parts counted in, and above bit 16 those whose CTA will not wait.
constexpr unsigned kCountMask = 0xFFFFu, kWontWait = 0x10000u;

// What a CTA joins of an item it shares.
enum : int { kJoinNothing = 0, kJoinShare = 1, kJoinAll = 2 };

// What a CTA adds to an item's count with its part.  It waits for the others
// only if all CTAs had begun at this count and at those before (waits).  The
// mark says what it will do, not what it found at this count: the two differ
// where the last CTA began between its counts of two items.
W4_RULE unsigned part_mark(bool all_begun, bool &waits) {
    waits = waits && all_begun;
    return 1u + (waits ? 0u : kWontWait);
}

// Looks at a count until `parts` are in it or `limit` ns are over; the count as last seen.
template <class Load, class Clock>
W4_RULE unsigned await_count(unsigned parts, uint64_t limit, Load load, Clock clock) {
    uint64_t t0 = 0;
    for (uint32_t spin = 0;; ++spin) {
        const unsigned now = load();
        if ((now & kCountMask) >= parts) return now;
        if ((spin & 63) == 63) {
            const uint64_t t = clock();
            if (t0 == 0) t0 = t;
            if (t - t0 > limit) return now;
        }
    }
}

// What a CTA joins that counted its part in as the count became `seen`, and,
// where it waits, saw `now` last (else `now` is `seen`).  Of parts that all
// wait, each CTA joins its share; else the last to count joins all.  `failed`:
// a wait ran out, or there are more counts than parts (a workspace that was
// not zeroed).
W4_RULE int join_mode(unsigned now, unsigned seen, bool waits, unsigned parts, bool &failed) {
    failed = false;
    if (waits && (now & kCountMask) == parts && now < kWontWait) return kJoinShare;
    if ((now & kCountMask) > parts || (now >> 16) > parts || (waits && (now & kCountMask) < parts)) {
        failed = true;
        return kJoinNothing;
    }
    if ((seen & kCountMask) != parts) return kJoinNothing;
    return seen < kWontWait ? kJoinShare : kJoinAll;
}

}  // namespace w4a16
