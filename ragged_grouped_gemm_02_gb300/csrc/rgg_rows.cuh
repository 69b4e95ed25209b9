// rgg_rows.cuh -- what the kernels that move rows between tokens and experts
// share: items of a row that a warp takes, and the choices' rows.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "rgg_ptx.cuh"

namespace rgg {

constexpr int kRowThreads = 256;
constexpr int kRowStatusBadIndex = 7;  // RGG_ERR_BAD_ROW_INDEX

// Warp-sized items over [T] tokens by `segs` segments of a row, in a grid-stride walk.
struct RowItems {
    int64_t item, step, items;
    int32_t segs;

    __device__ __forceinline__ RowItems(int64_t T, int32_t segs_) : segs(segs_) {
        item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
        step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
        items = T * segs_;
    }
    __device__ __forceinline__ bool left() const { return item < items; }
    __device__ __forceinline__ void next() { item += step; }
    __device__ __forceinline__ int64_t token() const {
        return items < (int64_t(1) << 32)
                   ? static_cast<int64_t>(static_cast<uint32_t>(item) / static_cast<uint32_t>(segs))
                   : item / segs;
    }
};

// The row of a choice as the kernels use it: -1 where it has none, and where the
// index is past the last row, which is recorded.
__device__ __forceinline__ int32_t checked_row(int32_t p, int64_t rows, int32_t* status) {
    if (p >= rows) {
        atomicCAS(status, 0, kRowStatusBadIndex);
        return -1;
    }
    return p < 0 ? -1 : p;
}

// Blocks of `threads` threads whose warps take `items` items, at most 2^30 (the walk strides by the grid).
inline int row_grid(int64_t items, int threads) {
    const int64_t warps = threads / 32, blocks = (items + warps - 1) / warps;
    return static_cast<int>(blocks < 1 ? 1 : (blocks > (int64_t(1) << 30) ? (int64_t(1) << 30) : blocks));
}

}  // namespace rgg
