// gmm_grid.h - the number of workgroups of a kernel that strides over its work. Plain arithmetic,
// the same on the host, where it is tested.
#pragma once
#include <stdint.h>

namespace gmm {

// Workgroups of `threads` for `items` pieces of work, one each or, beyond the limit, in turns: a
// launch of 2^32 threads in x or more is refused.
constexpr unsigned grid_for(int64_t items, int threads) {
    const int64_t most = ((int64_t)1 << 30) / threads;
    return (unsigned)(items < most ? items : most);
}

}  // namespace gmm
