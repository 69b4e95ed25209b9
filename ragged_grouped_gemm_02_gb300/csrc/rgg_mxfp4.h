// rgg_mxfp4.h -- the MXFP4 layouts shared by the quantisers and the product.
//
// Codes: two E2M1 values a byte, the even K index in the low half, K
// contiguous: [rows, K / 2].  Scales: one E8M0 byte (2^(byte - 127)) per 32
// values along K, in blocks of 128 rows by 4 scales (128 values of K), 512
// bytes each, the order the tensor core's scale memory takes them in: row r and
// scale s of a block at (r % 32) * 16 + (r / 32) * 4 + s.  The blocks of 128
// rows follow each other along K first: [row block, ceil(K / 128), 512].
//
// Row blocks start at the first row of an expert, so that a tile of 128 rows
// reads whole blocks.  For activations the first block of expert e is
// off[e] / 128 + e: experts then never share a block, whatever their counts
// (floor((a + m) / 128) - floor(a / 128) + 1 >= ceil(m / 128)), no prefix sum is
// needed, and M_tot / 128 + E blocks hold every routing of M_tot rows.  For
// weights [E, N, K] it is e * ceil(N / 128).
#pragma once

#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace rgg {

constexpr int kMxBlock = 32;        // values of K per scale
constexpr int kMxRows = 128;        // rows per block of scales
constexpr int kMxBlockBytes = 512;  // 128 rows by 4 scales
constexpr int kMxNan = 255;         // E8M0 NaN

__host__ __device__ inline int64_t mx_k_blocks(int64_t K) { return (K + 127) / 128; }
// The row block that row `r` of expert e (which starts at row `first` of all) is in.
__host__ __device__ inline int64_t mx_row_block(int64_t first, int e, int64_t r) { return first / kMxRows + e + r / kMxRows; }
__host__ __device__ inline int64_t mx_row_blocks(int64_t M_tot, int E) { return M_tot / kMxRows + E; }
// The place of row `r` of its block (0 <= r < 128) and its first scale.
__host__ __device__ inline int mx_in_block(int r) { return (r % 32) * 16 + (r / 32) * 4; }

}  // namespace rgg
