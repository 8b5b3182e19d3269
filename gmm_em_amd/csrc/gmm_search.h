// gmm_search.h - the steps of a search in sorted keys, four probes at a time (gmm_embed.hip). Plain
// arithmetic, the same on the host, where it is tested.
#pragma once
#include <stdint.h>

namespace gmm {

// Looks for the first of n sorted keys that is not below some key c. It lies in [lo, hi]; lo == hi ends
// the search. Searches that share a loop end after different numbers of steps: one that has
// ended has no probe inside and stays as it is.
struct Search {
    int64_t lo, hi;
    constexpr int64_t step() const { return (hi - lo + 4) / 5; }
    // place of probe q = 0 .. 3; its key is read only where it lies inside
    constexpr int64_t place(int q) const { return lo + (q + 1) * step() - 1; }
    constexpr bool inside(int64_t at) const { return at >= lo && at < hi; }
    // the first `below` probes have keys below c
    constexpr void narrow(int below) {
        if (lo == hi) return;
        const int64_t s = step();
        lo += below * s;
        if (below < 4 && lo + s - 1 < hi) hi = lo + s - 1;  // (the place behind the fourth was not seen)
    }
};

}  // namespace gmm
