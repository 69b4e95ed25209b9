// rgg_wgrad_parts.h -- the parts that the weight gradient splits an expert's
// rows into (rgg_wgrad.cuh).  Plain arithmetic, also for the host.
#pragma once

#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace rgg {

constexpr int kWgradRows = 64;  // rows (reduction) per stage

struct WgradPart {
    int32_t first, rows;  // rows [first, first + rows) of the expert's
};

// Part `part` of `split` of an expert's m rows: an equal share, rounded up to
// whole stages; the last parts may be short or empty.  An expert may have up to
// 2^31 - 1 rows, so the sums are unsigned: m + split - 1 and part * share, below
// m + 64 * split, pass 2^31 but not 2^32.
__host__ __device__ inline WgradPart wgrad_part(int32_t m, int32_t split, int32_t part) {
    const uint32_t all = static_cast<uint32_t>(m), parts = static_cast<uint32_t>(split);
    const uint32_t share = ((all + parts - 1u) / parts + kWgradRows - 1u) / kWgradRows * kWgradRows;
    const uint32_t from = static_cast<uint32_t>(part) * share;
    const uint32_t first = from < all ? from : all;
    const uint32_t left = all - first;
    return WgradPart{static_cast<int32_t>(first), static_cast<int32_t>(left < share ? left : share)};
}

}  // namespace rgg
