// pages_plan.h -- how many CTAs idx_pages_update's cluster has. Host code without CUDA, so that it can be tried with a
// device that has no room for a wide cluster.
#pragma once

#include <stdint.h>

namespace idx {

constexpr int kCtas = 8, kCtasMost = 16;
// Table entries and pages above which a wide cluster is taken. Replayed, eight CTAs / sixteen: 12,000 11.4 / 11.0 us, 39,000 of
// rows 13.1 / 12.6 and of pages 12.0 / 12.1, 76,000 15.6 / 14.4, 95,000 15.2 / 15.1, 100,000 of pages 14.2 / 12.6, 150,000 15.5 /
// 14.4, 301,000 20.3 / 17.1, 668,000 34.0 / 23.3, 1,010,000 45.7 / 28.2: below it sixteen gain up to 1.6 us, with twice the SMs.
constexpr int64_t kMany = 100000;

// wide_clusters(): how many clusters of kCtasMost CTAs the device takes at once; negative or 0 where it takes none, or where
// asking failed. Not every GPU, or part of one, has sixteen free SMs in one place; eight CTAs do the same work.
template <typename Query>
inline int pages_ctas(int64_t entries, Query wide_clusters) {
    return entries > kMany && wide_clusters() > 0 ? kCtasMost : kCtas;
}

}  // namespace idx
