// Checks gmm_grid.h: every launch has fewer than 2^32 threads, one workgroup at least, and as many as there
// are pieces of work where that is allowed by far.
#include <cstdint>
#include <cstdio>

#include "gmm_grid.h"

int main() {
    for (int threads = 64; threads <= 1024; threads += 64)
        for (int bit = 0; bit <= 40; ++bit)
            for (int64_t off = -2; off <= 2; ++off) {
                const int64_t items = (int64_t(1) << bit) + off;
                if (items < 1) continue;
                const int64_t grid = gmm::grid_for(items, threads);
                const bool few = items * threads <= int64_t(1) << 30;
                if (grid < 1 || grid > items || grid * threads >= int64_t(1) << 32 || (few && grid != items)) {
                    std::printf("%lld items of %d threads: %lld workgroups\n", (long long)items, threads,
                                (long long)grid);
                    return 1;
                }
            }
    std::puts("ok");
    return 0;
}
