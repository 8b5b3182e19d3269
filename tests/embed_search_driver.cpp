// Runs the search of gmm_search.h for numbers of keys n and every first place t (or many of them), as
// a wave does: 16 searches share a loop that goes on until the last has ended. Exits with 1 and
// says so if a probe's place is not one of the n keys or a search ends at another place than t.
//
// A search's probes depend on its keys only by t: a place has a key below c where it is before t.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gmm_search.h"

using gmm::Search;

static int fail(const char* what, int64_t n, int64_t t, int64_t at) {
    std::printf("%s: n %lld, first place %lld, at %lld\n", what, (long long)n, (long long)t, (long long)at);
    return 1;
}

static int check(int64_t n, int64_t stride, int extra) {
    for (int64_t t = 0; t <= n; t += (t < 64 || t + 64 > n) ? 1 : stride) {
        Search s{0, n};
        int steps = 0;
        // `extra`: steps that others of the wave still take
        for (int more = 0; s.lo < s.hi || more++ < extra;) {
            int below = 0;
            for (int q = 0; q < 4; ++q) {
                const int64_t at = s.place(q);
                if (!s.inside(at)) continue;
                if (at < 0 || at >= n) return fail("a key out of range", n, t, at);
                below += at < t;
            }
            s.narrow(below);
            if (++steps > 100) return fail("no end", n, t, s.lo);
        }
        if (s.lo != t) return fail("another place", n, t, s.lo);
    }
    return 0;
}

int main(int argc, char** argv) {
    const int extra = argc > 1 ? std::atoi(argv[1]) : 8;
    // few keys, wholly
    for (int64_t n = 0; n <= 700; ++n)
        if (check(n, 1, extra)) return 1;
    // about the powers of five, where searches of one wave need different numbers of steps
    for (int64_t p = 625; p <= 9765625; p *= 5)
        for (int64_t n : {p - 1, p, p + 1, p * 21 / 20, p * 5 / 4 - 1, p * 5 / 4, p * 5 / 4 + 1})
            if (check(n, n > 200000 ? n / 1009 : 1, extra)) return 1;
    // sizes in between
    for (int64_t n = 4097; n <= 100000; n += 61)
        if (check(n, 29, extra)) return 1;
    // the most rows of a gradient
    for (int64_t n : {int64_t(0x7fffffff), int64_t(1) << 30, int64_t(1220703125), int64_t(1525878906)})
        if (check(n, n / 100003, extra)) return 1;
    std::puts("ok");
    return 0;
}
