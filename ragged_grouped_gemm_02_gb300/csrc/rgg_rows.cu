// rgg_rows.cu -- rows of tokens to rows of experts and back.
//
//     dispatch   Xs[position[t, j]] = X[t]
//     combine    out[t] = sum over j of w[t, j] * Y[position[t, j]]
//     combine's gradient   dY[position[t, j]] = w[t, j] * dout[t]
//                          dw[t, j] = sum over columns of dout[t] * Y[position[t, j]]
//
// All of them go by token, so a token's row is read (or written) once however many
// experts it went to, and sums over its choices are made in registers, in the order
// of the choices: no atomics, equal calls give equal bits.  Choices without a row
// (position -1) add nothing; rows of no choice are left alone.  Bound by memory.
//
// A warp takes a token and a part of its row; the widest loads and stores that the
// row's size and the pointers' alignment allow.
#include <cuda_bf16.h>

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_rows.cuh"

namespace rgg {

constexpr int kDispatchLoads = 4;  // in flight a lane
constexpr int kCombineCols = 8;    // columns a lane
constexpr int kCombineSeg = 32 * kCombineCols;
constexpr int kGradThreads = 128;
constexpr int kGradChoices = 8;    // choices whose sums a thread holds at a time

// V: uint4, uint2, uint32_t, uint16_t or uint8_t; row_v: a row in those.
template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const V* __restrict__ X, const int32_t* __restrict__ position, int64_t T, int k, int64_t row_v,
                    int64_t rows, V* __restrict__ out, int32_t* status) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t segs = static_cast<int32_t>((row_v + 32 * kDispatchLoads - 1) / (32 * kDispatchLoads));
    for (RowItems it(T, segs); it.left(); it.next()) {
        const int64_t t = it.token();
        const int64_t c = (it.item - t * segs) * (32 * kDispatchLoads) + lane;
        V v[kDispatchLoads];
#pragma unroll
        for (int u = 0; u < kDispatchLoads; ++u)
            if (c + 32 * u < row_v) v[u] = X[t * row_v + c + 32 * u];
        for (int j = 0; j < k; ++j) {
            const int32_t p = checked_row(position[t * k + j], rows, status);
            if (p < 0) continue;
#pragma unroll
            for (int u = 0; u < kDispatchLoads; ++u)
                if (c + 32 * u < row_v) out[p * row_v + c + 32 * u] = v[u];
        }
    }
}

// kVec bf16 values in a load or store.
template <int kVec>
struct Bf16Vec;
template <>
struct Bf16Vec<8> {
    using type = uint4;
};
template <>
struct Bf16Vec<4> {
    using type = uint2;
};
template <>
struct Bf16Vec<2> {
    using type = uint32_t;
};
template <>
struct Bf16Vec<1> {
    using type = uint16_t;
};

template <int kVec>
__device__ __forceinline__ void bf16_values(const typename Bf16Vec<kVec>::type& v, float* x) {
    if constexpr (kVec == 1) {
        x[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <int kVec>
__device__ __forceinline__ typename Bf16Vec<kVec>::type bf16_pack(const float* x) {
    typename Bf16Vec<kVec>::type v;
    if constexpr (kVec == 1) {
        v = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) w[i] = pack_bf16x2(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]));
    }
    return v;
}

template <int kVec>
__global__ void __launch_bounds__(kRowThreads)
    combine_kernel(const __nv_bfloat16* __restrict__ Y, const int32_t* __restrict__ position,
                   const float* __restrict__ weights, int64_t T, int k, int64_t rows, int64_t N,
                   __nv_bfloat16* __restrict__ out, int32_t* status) {
    using V = typename Bf16Vec<kVec>::type;
    constexpr int kLoads = kCombineCols / kVec;
    constexpr int kFlight = 4;  // choices whose loads are in flight together
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t segs = static_cast<int32_t>((N + kCombineSeg - 1) / kCombineSeg);
    for (RowItems it(T, segs); it.left(); it.next()) {
        const int64_t t = it.token();
        const int64_t c = (it.item - t * segs) * kCombineSeg + lane * kVec;
        float acc[kCombineCols];
#pragma unroll
        for (int i = 0; i < kCombineCols; ++i) acc[i] = 0.0f;
        for (int k0 = 0; k0 < k; k0 += 32) {
            int32_t p = -1;  // lane j: choice k0 + j
            float w = 0.0f;
            if (k0 + lane < k) {
                p = checked_row(position[t * k + k0 + lane], rows, status);
                w = weights ? weights[t * k + k0 + lane] : 1.0f;
            }
            const int here = min(32, k - k0);
            for (int j0 = 0; j0 < here; j0 += kFlight) {
                V v[kFlight][kLoads];
                int32_t pj[kFlight];
#pragma unroll
                for (int j = 0; j < kFlight; ++j) {
                    pj[j] = __shfl_sync(0xffffffffu, p, (j0 + j) & 31);
                    if (j0 + j >= here) pj[j] = -1;
                    if (pj[j] < 0) continue;
                    const __nv_bfloat16* row = Y + pj[j] * N;
#pragma unroll
                    for (int u = 0; u < kLoads; ++u)
                        if (c + 32 * kVec * u < N) v[j][u] = *reinterpret_cast<const V*>(row + c + 32 * kVec * u);
                }
#pragma unroll
                for (int j = 0; j < kFlight; ++j) {
                    const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                    if (pj[j] < 0) continue;
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        if (c + 32 * kVec * u >= N) continue;
                        float x[kVec];
                        bf16_values<kVec>(v[j][u], x);
#pragma unroll
                        for (int i = 0; i < kVec; ++i) acc[u * kVec + i] += wj * x[i];
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            if (c + 32 * kVec * u < N)
                *reinterpret_cast<V*>(out + t * N + c + 32 * kVec * u) = bf16_pack<kVec>(acc + u * kVec);
    }
}

// A block takes a token: its threads walk the columns and hold their parts of the
// choices' sums, which the block then adds in a fixed order.
template <int kVec>
__global__ void __launch_bounds__(kGradThreads)
    combine_backward_kernel(const __nv_bfloat16* __restrict__ dout, const __nv_bfloat16* __restrict__ Y,
                            const int32_t* __restrict__ position, const float* __restrict__ weights, int64_t T, int k,
                            int64_t rows, int64_t N, __nv_bfloat16* __restrict__ dY, float* __restrict__ dweights,
                            int32_t* status) {
    using V = typename Bf16Vec<kVec>::type;
    __shared__ float s_part[kGradThreads / 32][kGradChoices];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int k0 = 0; k0 < k; k0 += kGradChoices) {
            int32_t p[kGradChoices];
            float w[kGradChoices], sum[kGradChoices];
#pragma unroll
            for (int j = 0; j < kGradChoices; ++j) {
                p[j] = k0 + j < k ? checked_row(position[t * k + k0 + j], rows, status) : -1;
                w[j] = p[j] >= 0 ? weights[t * k + k0 + j] : 0.0f;
                sum[j] = 0.0f;
            }
            for (int64_t c = static_cast<int64_t>(threadIdx.x) * kVec; c < N; c += kGradThreads * kVec) {
                float d[kVec];
                bf16_values<kVec>(*reinterpret_cast<const V*>(dout + t * N + c), d);
                V v[kGradChoices];
#pragma unroll
                for (int j = 0; j < kGradChoices; ++j)
                    if (p[j] >= 0) v[j] = *reinterpret_cast<const V*>(Y + p[j] * N + c);
#pragma unroll
                for (int j = 0; j < kGradChoices; ++j) {
                    if (p[j] < 0) continue;
                    float y[kVec], g[kVec];
                    bf16_values<kVec>(v[j], y);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        sum[j] += d[i] * y[i];
                        g[i] = w[j] * d[i];
                    }
                    if (dY) *reinterpret_cast<V*>(dY + p[j] * N + c) = bf16_pack<kVec>(g);
                }
            }
            if (!dweights) continue;
#pragma unroll
            for (int j = 0; j < kGradChoices; ++j) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], s);
                if (lane == 0) s_part[warp][j] = sum[j];
            }
            __syncthreads();
            if (threadIdx.x < kGradChoices && k0 + static_cast<int>(threadIdx.x) < k) {
                float all = 0.0f;
#pragma unroll
                for (int i = 0; i < kGradThreads / 32; ++i) all += s_part[i][threadIdx.x];
                dweights[t * k + k0 + threadIdx.x] = all;
            }
            __syncthreads();
        }
    }
}

template <typename V>
static cudaError_t launch_dispatch(const void* X, const int32_t* position, int64_t T, int k, int64_t row_bytes,
                                   int64_t rows, void* out, int32_t* status, cudaStream_t st) {
    const int64_t row_v = row_bytes / static_cast<int64_t>(sizeof(V));
    const int64_t segs = (row_v + 32 * kDispatchLoads - 1) / (32 * kDispatchLoads);
    return launch_chained(dispatch_kernel<V>, row_grid(T * segs, kRowThreads), kRowThreads, 0, st,
                          static_cast<const V*>(X), position, T, k, row_v, rows, static_cast<V*>(out), status);
}

// The widest of 16, 8, 4, 2 and 1 bytes that divides a row and all addresses.
static int common_width(int64_t row_bytes, std::initializer_list<const void*> p) {
    uintptr_t all = static_cast<uintptr_t>(row_bytes) | 16u;
    for (const void* q : p) all |= reinterpret_cast<uintptr_t>(q);
    return static_cast<int>(all & (~all + 1));
}

// 0 <= T, rows < 2^31, 1 <= k, 1 <= row < 2^31.
static bool rows_ok(int64_t T, int k, int64_t rows, int64_t row) {
    const int64_t most = int64_t(1) << 31;
    return T >= 0 && T < most && rows >= 0 && rows < most && k >= 1 && row >= 1 && row < most && T * k < most;
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
    cudaError_t err;
    switch (common_width(row_bytes, {X, out})) {
        case 16: err = launch_dispatch<uint4>(X, position, T, k, row_bytes, rows, out, dev.status, st); break;
        case 8: err = launch_dispatch<uint2>(X, position, T, k, row_bytes, rows, out, dev.status, st); break;
        case 4: err = launch_dispatch<uint32_t>(X, position, T, k, row_bytes, rows, out, dev.status, st); break;
        case 2: err = launch_dispatch<uint16_t>(X, position, T, k, row_bytes, rows, out, dev.status, st); break;
        default: err = launch_dispatch<uint8_t>(X, position, T, k, row_bytes, rows, out, dev.status, st); break;
    }
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "dispatch launch");
}

extern "C" rgg_status rgg_combine(rgg_handle* h, const void* Y, const int32_t* position, const float* weights, int64_t T,
                                  int k, int64_t rows, int64_t N, void* out, void* stream) {
    if (!h || !rows_ok(T, k, rows, N)) return RGG_ERR_INVALID_ARG;
    if (T == 0) return RGG_OK;
    if ((rows > 0 && !Y) || !position || !out || !host_aligned(position, 4) || !host_aligned(weights, 4) ||
        !host_aligned(Y, 2) || !host_aligned(out, 2))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int width = common_width(2 * N, {Y, out});
    const int grid = row_grid(T * ((N + kCombineSeg - 1) / kCombineSeg), kRowThreads);
    auto kernel = width == 16 ? combine_kernel<8> : width == 8 ? combine_kernel<4>
                  : width == 4 ? combine_kernel<2> : combine_kernel<1>;
    cudaError_t err = launch_chained(kernel, grid, kRowThreads, 0, st, static_cast<const __nv_bfloat16*>(Y), position,
                                     weights, T, k, rows, N, static_cast<__nv_bfloat16*>(out), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "combine launch");
}

extern "C" rgg_status rgg_combine_backward(rgg_handle* h, const void* dout, const void* Y, const int32_t* position,
                                           const float* weights, int64_t T, int k, int64_t rows, int64_t N, void* dY,
                                           float* dweights, void* stream) {
    if (!h || !rows_ok(T, k, rows, N)) return RGG_ERR_INVALID_ARG;
    if (T == 0 || (!dY && !dweights)) return RGG_OK;
    if (!dout || (rows > 0 && !Y) || !position || !weights || !host_aligned(position, 4) || !host_aligned(weights, 4) ||
        !host_aligned(dweights, 4) || !host_aligned(dout, 2) || !host_aligned(Y, 2) || !host_aligned(dY, 2))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int width = common_width(2 * N, {dout, Y, dY});
    auto kernel = width == 16 ? combine_backward_kernel<8> : width == 8 ? combine_backward_kernel<4>
                  : width == 4 ? combine_backward_kernel<2> : combine_backward_kernel<1>;
    cudaError_t err = launch_chained(kernel, static_cast<int>(T), kGradThreads, 0, st,
                                     static_cast<const __nv_bfloat16*>(dout), static_cast<const __nv_bfloat16*>(Y),
                                     position, weights, T, k, rows, N, static_cast<__nv_bfloat16*>(dY), dweights, dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "combine_backward launch");
}
