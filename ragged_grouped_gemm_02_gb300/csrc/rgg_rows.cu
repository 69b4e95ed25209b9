// rgg_rows.cu -- rows of tokens to rows of experts and back.
//
//     dispatch   Xs[position[t, j]] = X[t]
//     combine    out[t] = sum over j of w[t, j] * Y[position[t, j]]
//     combine's gradient   dY[position[t, j]] = w[t, j] * dout[t]
//                          dw[t, j] = sum over columns of dout[t] * Y[position[t, j]]
//
// Dispatch and combine go by token: a token's row comes from memory (or goes there)
// once however many experts it went to, and sums over its choices are made in registers, in
// the order of the choices.  Combine's gradient goes by choice; the choices of a token are
// neighbours, so that dout's row comes from memory once and from cache k - 1 times, as X's does in
// dispatch where rows are not whole 16 bytes.  No atomics, equal calls give equal bits.  Choices without a row
// (position -1) add nothing; rows of no choice are left alone.  Bound by memory.
//
// Rows move in blocks of 16 bytes, aligned where they are written.  Where rows are not
// whole 16 bytes (an odd width), a block that is read starts anywhere: it is put together
// from an aligned one and the next lane's, by a funnel shift that is the same for a whole
// row (so 32 lanes give 31 blocks); the first and last blocks of a written row are stored
// element by element.  A row that is read next to a tensor's end, where the blocks around it may
// be outside, is read byte by byte over its whole length.
//
// Measured: 8,192 tokens x 4, 6144 columns (503 MB) dispatch 75 us, combine 81, its gradient (906 MB)
// 135; 8,192 x 6 of 2688 columns 47, 53 and 93, of 2693 columns 57, 83 and 123, where
// element-wise loads and stores took 91, 141 and 277.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_rows.cuh"

namespace rgg {

constexpr int kDispatchLoads = 2;  // in flight a lane
constexpr int kFlight = 2;         // choices whose loads are in flight together
constexpr int kCombineSteps = 2;   // blocks that a lane combines at a time

// A tensor's bytes, for loads that may not leave them.
struct Span {
    uintptr_t begin, end;
};

// The 16 bytes at `at`, those outside the span 0.  For the few rows at a tensor's ends: a call, so that the
// other rows' code has the registers to itself.
__device__ __noinline__ uint4 load_edge(uintptr_t at, uintptr_t begin, uintptr_t end) {
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int i = 15; i >= 0; --i) {
        hi = (hi << 8) | (lo >> 56);
        lo <<= 8;
        if (at + i >= begin && at + i < end) lo |= *reinterpret_cast<const uint8_t*>(at + i);
    }
    return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                      static_cast<uint32_t>(hi >> 32));
}

// How a block of 16 bytes is read: aligned; from an aligned one and the next lane's; byte by
// byte, where those may be outside the tensor.
constexpr int kAligned = 0, kShifted = 1, kEdge = 2;

template <int kMode>
__device__ __forceinline__ uint4 load_block(uintptr_t at, Span in) {
    if constexpr (kMode == kEdge) return load_edge(at, in.begin, in.end);
    else return __ldg(reinterpret_cast<const uint4*>(kMode == kShifted ? at & ~static_cast<uintptr_t>(15) : at));
}
// Whether the aligned blocks around a row are inside the tensor: all that a lane loads of it, or the lane before it needs.
__device__ __forceinline__ bool row_inside(uintptr_t row, int32_t bytes, Span in) {
    return row >= in.begin + 32 && row + bytes + 48 <= in.end;
}
// kShifted: the 16 bytes that start `shift` bytes (the same in all lanes) into v, the next lane's v behind it.  Whole warp.
template <int kMode>
__device__ __forceinline__ uint4 shift_block(const uint4& v, uint32_t shift) {
    if constexpr (kMode != kShifted) return v;
    const uint32_t bits = 8 * (shift & 3);
    auto next = [](uint32_t w) { return __shfl_down_sync(0xffffffffu, w, 1); };
    auto take = [&](uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t w4) {
        return make_uint4(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits), __funnelshift_r(w2, w3, bits),
                          __funnelshift_r(w3, w4, bits));
    };
    switch (shift >> 2) {
        case 0: return shift == 0 ? v : take(v.x, v.y, v.z, v.w, next(v.x));
        case 1: return take(v.y, v.z, v.w, next(v.x), next(v.y));
        case 2: return take(v.z, v.w, next(v.x), next(v.y), next(v.z));
        default: return take(v.w, next(v.x), next(v.y), next(v.z), next(v.w));
    }
}
// Blocks that a warp's lanes give.
__host__ __device__ constexpr int block_lanes(bool whole) { return whole ? 32 : 31; }

// The aligned blocks of a row [row, row + bytes): the b-th starts `at(b)` bytes into it (the first may be before it).
// Rows are shorter than 2^30 bytes, so that places in them are 32-bit numbers.
constexpr int64_t kRowBytes = int64_t(1) << 30;
struct RowBlocks {
    int32_t bytes, lead;
    __device__ __forceinline__ RowBlocks(uintptr_t row, int32_t bytes_) : bytes(bytes_), lead(static_cast<int32_t>(row & 15)) {}
    __device__ __forceinline__ int32_t count() const { return (bytes + lead + 15) / 16; }
    __device__ __forceinline__ int32_t at(int32_t b) const { return 16 * b - lead; }
    __device__ __forceinline__ bool whole(int32_t off) const { return off >= 0 && off + 16 <= bytes; }
};
inline __host__ __device__ int32_t most_blocks(int32_t bytes, bool aligned) { return aligned ? bytes / 16 : (bytes + 15) / 16 + 1; }

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Eight values, rounded, to the block `off` bytes into a row; a block that is not whole element by element.
template <int kMode>
__device__ __forceinline__ void store8(uintptr_t row, int32_t off, const RowBlocks& blocks, const float (&x)[8]) {
    const uint32_t w[4] = {pack_bf16x2(__float_as_uint(x[0]), __float_as_uint(x[1])),
                           pack_bf16x2(__float_as_uint(x[2]), __float_as_uint(x[3])),
                           pack_bf16x2(__float_as_uint(x[4]), __float_as_uint(x[5])),
                           pack_bf16x2(__float_as_uint(x[6]), __float_as_uint(x[7]))};
    if (kMode == kAligned || blocks.whole(off)) {
        *reinterpret_cast<uint4*>(row + off) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (kMode != kAligned) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (off + 2 * i >= 0 && off + 2 * i < blocks.bytes)
                *reinterpret_cast<uint16_t*>(row + off + 2 * i) = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

template <bool kWhole>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(uintptr_t X, const int32_t* __restrict__ position, int64_t T, int k, int32_t row_bytes, int64_t rows,
                    uintptr_t out, int32_t* status) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    constexpr int kLanes = block_lanes(kWhole);
    const int32_t most = most_blocks(row_bytes, kWhole);
    const int32_t segs = (most + kLanes * kDispatchLoads - 1) / (kLanes * kDispatchLoads);
    const Span span{X, X + T * row_bytes};
    for (RowItems it(T, segs); it.left(); it.next()) {
        const int64_t t = it.token();
        const int32_t b0 = static_cast<int32_t>(it.item - t * segs) * (kLanes * kDispatchLoads) + lane;
        const uintptr_t from = X + t * row_bytes;
        if constexpr (kWhole) {
            uint4 v[kDispatchLoads];
#pragma unroll
            for (int u = 0; u < kDispatchLoads; ++u)
                if (b0 + 32 * u < most) v[u] = __ldg(reinterpret_cast<const uint4*>(from) + b0 + 32 * u);
            for (int j = 0; j < k; ++j) {
                const int32_t p = checked_row(position[t * k + j], rows, status);
                if (p < 0) continue;
                uint4* to = reinterpret_cast<uint4*>(out + static_cast<int64_t>(p) * row_bytes) + b0;
#pragma unroll
                for (int u = 0; u < kDispatchLoads; ++u)
                    if (b0 + 32 * u < most) to[32 * u] = v[u];
            }
        } else {
            auto copy = [&](auto mode, int32_t p) {
                constexpr int kMode = decltype(mode)::value;
                const uintptr_t to = out + static_cast<int64_t>(p) * row_bytes;
                const RowBlocks blocks(to, row_bytes);
                const uint32_t shift = static_cast<uint32_t>(from - blocks.lead) & 15u;
                const int32_t count = blocks.count();
                uint4 v[kDispatchLoads];
#pragma unroll
                for (int u = 0; u < kDispatchLoads; ++u) {
                    v[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (b0 + kLanes * u <= count) v[u] = load_block<kMode>(from + blocks.at(b0 + kLanes * u), span);
                }
#pragma unroll
                for (int u = 0; u < kDispatchLoads; ++u) {
                    const int32_t off = blocks.at(b0 + kLanes * u);
                    const uint4 x = shift_block<kMode>(v[u], shift);
                    if (lane == 31 || b0 + kLanes * u >= count) continue;
                    if (blocks.whole(off)) {
                        *reinterpret_cast<uint4*>(to + off) = x;
                    } else {
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (off + i >= 0 && off + i < row_bytes)
                                *reinterpret_cast<uint8_t*>(to + off + i) = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
                    }
                }
            };
            const bool inside = row_inside(from, row_bytes, span);
            for (int j = 0; j < k; ++j) {
                const int32_t p = checked_row(position[t * k + j], rows, status);
                if (p < 0) continue;
                if (inside) copy(std::integral_constant<int, kShifted>(), p);
                else copy(std::integral_constant<int, kEdge>(), p);
            }
        }
    }
}

// A warp takes two blocks a lane of a token's row.
template <bool kWhole>
__global__ void __launch_bounds__(kRowThreads, 4)
    combine_kernel(uintptr_t Y, const int32_t* __restrict__ position, const float* __restrict__ weights, int64_t T, int k,
                   int64_t rows, int32_t N, uintptr_t out, int32_t* status) {
    constexpr int kSteps = kCombineSteps, kLanes = block_lanes(kWhole);
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t bytes = 2 * N;
    const int32_t segs = (most_blocks(bytes, kWhole) + kLanes * kSteps - 1) / (kLanes * kSteps);
    const Span span{Y, Y + rows * bytes};
    for (RowItems it(T, segs); it.left(); it.next()) {
        const int64_t t = it.token();
        const uintptr_t to = out + t * bytes;
        const RowBlocks blocks(to, bytes);
        const int32_t count = blocks.count();
        const int32_t b0 = static_cast<int32_t>(it.item - t * segs) * (kLanes * kSteps) + lane;
        float acc[kSteps][8];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[s][i] = 0.0f;
        for (int k0 = 0; k0 < k; k0 += 32) {
            int32_t p = -1;  // lane j: choice k0 + j
            float w = 0.0f;
            if (k0 + lane < k) {
                p = checked_row(position[t * k + k0 + lane], rows, status);
                w = weights ? weights[t * k + k0 + lane] : 1.0f;
            }
            const int here = min(32, k - k0);
            bool inside = true;
            if constexpr (!kWhole) inside = __all_sync(0xffffffffu, p < 0 || row_inside(Y + static_cast<int64_t>(p) * bytes, bytes, span));
            auto add = [&](auto mode) {
                constexpr int kMode = decltype(mode)::value;
                for (int j0 = 0; j0 < here; j0 += kFlight) {
                    uint4 v[kFlight][kSteps];
                    int32_t pj[kFlight];
#pragma unroll
                    for (int j = 0; j < kFlight; ++j) {
                        pj[j] = __shfl_sync(0xffffffffu, p, (j0 + j) & 31);
                        if (j0 + j >= here) pj[j] = -1;
                        if (pj[j] < 0) continue;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s)
                            if (b0 + kLanes * s < count + (kWhole ? 0 : 1)) v[j][s] = load_block<kMode>(Y + static_cast<int64_t>(pj[j]) * bytes + blocks.at(b0 + kLanes * s), span);
                    }
#pragma unroll
                    for (int j = 0; j < kFlight; ++j) {
                        const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                        if (pj[j] < 0) continue;
                        const uint32_t shift = static_cast<uint32_t>(Y + static_cast<int64_t>(pj[j]) * bytes - blocks.lead) & 15u;
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            float x[8];
                            unpack8(shift_block<kMode>(v[j][s], shift), x);
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[s][i] += wj * x[i];
                        }
                    }
                }
            };
            if constexpr (kWhole) add(std::integral_constant<int, kAligned>());
            else if (inside) add(std::integral_constant<int, kShifted>());
            else add(std::integral_constant<int, kEdge>());
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if ((kWhole || lane < 31) && b0 + kLanes * s < count) store8<kWhole ? kAligned : kShifted>(to, blocks.at(b0 + kLanes * s), blocks, acc[s]);
    }
}

// A warp takes a choice and walks its row: the dot product in its lanes, added in a
// fixed order, and the scaled gradient.  The warps of a token's choices are neighbours, so
// its gradient comes from memory once.
template <bool kWhole>
__global__ void __launch_bounds__(kRowThreads, 4)
    combine_backward_kernel(uintptr_t dout, uintptr_t Y, const int32_t* __restrict__ position,
                            const float* __restrict__ weights, int64_t T, int k, int64_t rows, int32_t N, uintptr_t dY,
                            float* __restrict__ dweights, int32_t* status) {
    constexpr int kLoads = 3;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t bytes = 2 * N;
    const Span d_span{dout, dout + T * bytes}, y_span{Y, Y + rows * bytes};
    for (RowItems it(T, k); it.left(); it.next()) {
        const int64_t t = it.token();
        const int32_t p = checked_row(position[it.item], rows, status);
        float sum = 0.0f;
        if (p >= 0) {
            const float w = weights[it.item];
            const uintptr_t d_row = dout + t * bytes, y_row = Y + static_cast<int64_t>(p) * bytes, to = dY + static_cast<int64_t>(p) * bytes;
            const RowBlocks blocks(dY ? to : y_row, bytes);
            const uint32_t d_shift = static_cast<uint32_t>(d_row - blocks.lead) & 15u;
            const uint32_t y_shift = static_cast<uint32_t>(y_row - blocks.lead) & 15u;
            const int32_t count = blocks.count();
            auto walk = [&](auto d_mode, auto y_mode) {
                constexpr int kD = decltype(d_mode)::value, kY = decltype(y_mode)::value;
                constexpr int kLanes = block_lanes(kWhole);
                for (int32_t first = 0; first < count; first += kLanes * kLoads) {
                    const int32_t b0 = first + lane;
                    uint4 dv[kLoads], yv[kLoads];
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        dv[u] = yv[u] = make_uint4(0u, 0u, 0u, 0u);
                        const int32_t off = blocks.at(b0 + kLanes * u);
                        if (b0 + kLanes * u >= count + (kWhole ? 0 : 1)) continue;
                        yv[u] = load_block<kY>(y_row + off, y_span);
                        dv[u] = load_block<kD>(d_row + off, d_span);
                    }
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        const int32_t off = blocks.at(b0 + kLanes * u);
                        float d[8], y[8];
                        unpack8(shift_block<kD>(dv[u], d_shift), d);
                        unpack8(shift_block<kY>(yv[u], y_shift), y);
                        if ((!kWhole && lane == 31) || b0 + kLanes * u >= count) continue;
                        if (!kWhole && !blocks.whole(off)) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (off + 2 * i < 0 || off + 2 * i >= bytes) d[i] = y[i] = 0.0f;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            sum += d[i] * y[i];
                            d[i] *= w;
                        }
                        if (dY) store8<kWhole ? kAligned : kShifted>(to, off, blocks, d);
                    }
                }
            };
            using Shifted = std::integral_constant<int, kShifted>;
            using Aligned = std::integral_constant<int, kAligned>;
            using Edge = std::integral_constant<int, kEdge>;
            if constexpr (kWhole) walk(Aligned(), Aligned());
            else if (!row_inside(d_row, bytes, d_span) || !row_inside(y_row, bytes, y_span)) walk(Edge(), Edge());
            else if (y_shift == 0) walk(Shifted(), Aligned());  // dY and Y alike: its blocks are Y's own
            else walk(Shifted(), Shifted());
        }
        if (!dweights) continue;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) dweights[it.item] = sum;
    }
}

// Whether rows of that size at these addresses are whole, aligned 16 bytes.
static bool rows_aligned(int64_t row_bytes, std::initializer_list<const void*> p) {
    uintptr_t all = static_cast<uintptr_t>(row_bytes);
    for (const void* q : p) all |= reinterpret_cast<uintptr_t>(q);
    return (all & 15u) == 0;
}
static uintptr_t address(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// 0 <= T, rows, T k < 2^31, 1 <= k, 1 <= row_bytes < 2^30.
static bool rows_ok(int64_t T, int k, int64_t rows, int64_t row_bytes) {
    const int64_t most = int64_t(1) << 31;
    return T >= 0 && T < most && rows >= 0 && rows < most && k >= 1 && row_bytes >= 1 && row_bytes < kRowBytes && T * k < most;
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_dispatch(rgg_handle* h, const void* X, const int32_t* position, int64_t T, int k, int64_t rows,
                                   int64_t row_bytes, void* out, void* stream) {
    if (!h || !rows_ok(T, k, rows, row_bytes)) return RGG_ERR_INVALID_ARG;
    if (T == 0) return RGG_OK;
    if (!X || !position || (rows > 0 && !out) || !host_aligned(position, 4)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool aligned = rows_aligned(row_bytes, {X, out});
    const int32_t bytes = static_cast<int32_t>(row_bytes);
    const int64_t segs = (most_blocks(bytes, aligned) + block_lanes(aligned) * kDispatchLoads - 1) /
                         (block_lanes(aligned) * kDispatchLoads);
    cudaError_t err = launch_chained(aligned ? dispatch_kernel<true> : dispatch_kernel<false>,
                                     row_grid(T * segs, kRowThreads), kRowThreads, 0, st, address(X), position, T, k,
                                     bytes, rows, address(out), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "dispatch launch");
}

extern "C" rgg_status rgg_combine(rgg_handle* h, const void* Y, const int32_t* position, const float* weights, int64_t T,
                                  int k, int64_t rows, int64_t N, void* out, void* stream) {
    if (!h || !rows_ok(T, k, rows, N < kRowBytes ? 2 * N : N)) return RGG_ERR_INVALID_ARG;
    if (T == 0) return RGG_OK;
    if ((rows > 0 && !Y) || !position || !out || !host_aligned(position, 4) || !host_aligned(weights, 4) ||
        !host_aligned(Y, 2) || !host_aligned(out, 2))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool aligned = rows_aligned(2 * N, {Y, out});
    const int32_t width = static_cast<int32_t>(N);
    const int64_t segs = (most_blocks(2 * width, aligned) + block_lanes(aligned) * kCombineSteps - 1) /
                         (block_lanes(aligned) * kCombineSteps);
    cudaError_t err = launch_chained(aligned ? combine_kernel<true> : combine_kernel<false>, row_grid(T * segs, kRowThreads),
                                     kRowThreads, 0, st, address(Y), position, weights, T, k, rows, width, address(out),
                                     dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "combine launch");
}

extern "C" rgg_status rgg_combine_backward(rgg_handle* h, const void* dout, const void* Y, const int32_t* position,
                                           const float* weights, int64_t T, int k, int64_t rows, int64_t N, void* dY,
                                           float* dweights, void* stream) {
    if (!h || !rows_ok(T, k, rows, N < kRowBytes ? 2 * N : N)) return RGG_ERR_INVALID_ARG;
    if (T == 0 || (!dY && !dweights)) return RGG_OK;
    if (!dout || (rows > 0 && !Y) || !position || !weights || !host_aligned(position, 4) || !host_aligned(weights, 4) ||
        !host_aligned(dweights, 4) || !host_aligned(dout, 2) || !host_aligned(Y, 2) || !host_aligned(dY, 2))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool aligned = rows_aligned(2 * N, {dout, Y, dY});
    cudaError_t err = launch_chained(aligned ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                                     row_grid(T * k, kRowThreads), kRowThreads, 0, st, address(dout), address(Y), position,
                                     weights, T, k, rows, static_cast<int32_t>(N), address(dY), dweights, dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "combine_backward launch");
}
