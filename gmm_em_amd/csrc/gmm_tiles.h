// gmm_tiles.h - the choice of a product's workgroup tiles (gmm_gemm.h) on the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gmm_gemm.h"

namespace gmm {

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
inline int pad(int64_t k) { return (int)((k + GK - 1) / GK * GK); }
// Workgroup tiles: codes or dims by rows.
template <int ID>
struct Tile;
template <>
struct Tile<0> {
    static constexpr int BM = 256, BN = 256, WM = 2, WN = 4;
};
template <>
struct Tile<1> {
    static constexpr int BM = 192, BN = 256, WM = 2, WN = 4;
};
template <>
struct Tile<2> {
    static constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
};
template <>
struct Tile<3> {
    static constexpr int BM = 64, BN = 64, WM = 2, WN = 2;
};

// The tile and the split of the contracted axis that take least time by a
// model of it: rounds of workgroups over the chip, each of a fixed part and a
// part per step, and the writing and reading of a split's partial sums.
struct TileCost {
    int bm, bn, at_once;  // workgroups on the chip
    float per_step, fixed;  // microseconds
};

struct Choice {
    int tile, split;
};
inline Choice choose_tile(const TileCost* costs, int64_t m, int64_t n, int64_t steps, int max_split,
                          size_t split_bytes) {
    Choice best{0, 1};
    double least = 1e300;
    for (int t = 0; t < 4; ++t) {
        const TileCost& c = costs[t];
        const int64_t tiles = ((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn);
        for (int s = 1; s <= max_split && s <= steps; ++s) {
            if (s > 1 && (size_t)s * m * n * 4 > split_bytes) break;
            const int64_t rounds = (tiles * s + c.at_once - 1) / c.at_once;
            double us = rounds * (c.fixed + c.per_step * (double)((steps + s - 1) / s));
            if (s > 1) us += 4.0 + (double)m * n * 8 * s / 4.0e6;
            if (us < least) {
                least = us;
                best = Choice{t, s};
            }
        }
    }
    return best;
}
template <typename F>
inline void with_tile(int tile, F f) {
    switch (tile) {
        case 0: f(std::integral_constant<int, 0>()); break;
        case 1: f(std::integral_constant<int, 1>()); break;
        case 2: f(std::integral_constant<int, 2>()); break;
        default: f(std::integral_constant<int, 3>()); break;
    }
}

inline unsigned tile_grid(int mt, int nt) {
    return (unsigned)(((int64_t)mt * nt + 7) / 8 * 8);
}

}  // namespace gmm
