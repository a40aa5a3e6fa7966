// fp8_plan.h -- which kernel of fp8.cu takes a product, and how its contraction is split; plain C++, so that the rule
// can be asked on the host as well.
#pragma once

#include <stdint.h>

namespace csa2 {

// The contraction of the columns kernel split (by 2, 4 or 8), two blocks each at least: to about one CTA an SM, and up
// to two in clusters of 4 at most (64 tiles of 32 blocks: 14.5 us by 2, 12.6 by 4; 32 tiles: 7.5 us by 4, 8.2 by 8).
inline int fp8_cols_split(int64_t tiles, int nb) {
    int split = 1;
    while (split < 8 && nb >= split * 4 && tiles * split * 2 <= (split < 4 ? 296 : 160)) split *= 2;
    return split;
}

// Whether the rows of x lie along the columns of tensor memory (tiles of at most 64 of them) rather than on its lanes.
// Both kernels' time goes by the blocks that a CTA takes one after the other: 0.53 us a block with rows of x along the
// columns (two CTAs an SM, 64 rows each, the contraction split for few tiles), 0.57 us with them on the lanes (one CTA an
// SM, 128 rows x 256). Measured (us, columns / lanes): 128 x 2112 x 7168 13.7 / 34, 256 x 4096 x 4096 17.8 / 20,
// 777 x 4099 x 4112 47 / 26, 128 x 32768 x 4096 44 / 28.
inline bool fp8_by_columns(int64_t m, int64_t n, int k) {
    if (m <= 64) return true;
    const int nb = (k + 127) / 128;
    const int64_t tc = ((n + 127) / 128) * ((m + 63) / 64), tr = ((n + 255) / 256) * ((m + 127) / 128);
    const int split = fp8_cols_split(tc, nb);
    const int64_t cols = (tc * split + 295) / 296 * ((nb + split - 1) / split), rows = (tr + 147) / 148 * nb;
    return cols * 53 <= rows * 57;
}

}  // namespace csa2
