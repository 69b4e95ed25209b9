// rgg_fp8_block.h -- the 8-bit form with a scale per block of 128, as the
// quantisers write it and the product reads it.
//
// Codes: E4M3 bytes, K contiguous: [rows, K].  Scales: fp32, one per row and 128
// values along K for activations, [rows, ceil(K / 128)]; one per 128 rows and 128
// of K for weights, [E, ceil(N / 128), ceil(K / 128)].  A value is code * scale.
#pragma once

#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace rgg {

constexpr int kFpBlock = 128;        // values of K, and columns of a weight, that share a scale
constexpr float kFpMax = 448.0f;     // E4M3's largest value
// The least largest magnitude a block is scaled by, 2^-100: 448 / a stays inside
// fp32's normal range.  (Its scale is 2^-108.8.  The product multiplies a row's scale by
// a weight's first, in fp32: two of the least give 0, two above 2^64 Inf.)
constexpr float kFpLeast = 7.888609052210118e-31f;

__host__ __device__ inline int64_t fp_blocks(int64_t n) { return (n + kFpBlock - 1) / kFpBlock; }

}  // namespace rgg
