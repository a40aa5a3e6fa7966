// attend_plan.h -- over how many CTAs the paged attention splits a row; plain C++, so that the rule can be asked on the
// host as well.
#pragma once

#include <initializer_list>

namespace csa2 {

// The cluster of a row with `tiles` tiles, where `rows` rows are attended to; fits(size): how many clusters of that size the
// device holds at once (0: none, or it takes none of that size). A tile takes about 3.5 us, what surrounds a row's
// tiles 11 and the join 2, so a row's tiles go over as many CTAs as leave every row's cluster on the GPU at once: a second
// round of clusters costs more than the split gains.
template <typename Fits>
inline int paged_attend_split(int rows, int tiles, Fits&& fits) {
    if (tiles < 2) return 1;
    for (int size : {16, 8, 6, 5, 4, 3, 2}) {
        if (rows > fits(size)) continue;
        const int most = size < tiles ? size : tiles, each = (tiles + most - 1) / most;
        return (tiles + each - 1) / each;  // no smaller cluster has as few tiles per CTA
    }
    return 1;
}

}  // namespace csa2
