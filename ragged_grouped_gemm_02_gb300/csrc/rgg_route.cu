// rgg_route.cu -- the router of a mixture of experts: the k largest of a token's
// E logits, their weights, and the weights' gradient by the logits.
//
// With l the logits and C the choices,
//     softmax   s_i = exp(l_i) / sum over all j of exp(l_j)
//     sigmoid   s_i = 1 / (1 + exp(-l_i))
//     weight    w_i = s_i, or s_i / (sum over C of s_j + 1e-20), times `scale`.
// (With softmax the divided form is exp(l_i) / sum over C of exp(l_j): the other
// experts' logits drop out.)  Gradients, g the gradient by the weights:
//     softmax             dl_j = scale s_j ([j in C] g_j - sum over C of g_i s_i)
//     softmax, divided    dl_i = scale w_i (g_i - sum g_j w_j),  i in C, else 0
//     sigmoid             dl_i = scale g_i s_i (1 - s_i),        i in C, else 0
//     sigmoid, divided    dl_i = scale (g_i - sum g_j w_j) / (sum s_j + 1e-20) s_i (1 - s_i)
// with w before the scale.
//
// A warp takes a token; lane l holds the logits l, l + 32, ...  The order is by
// value, ties to the lower expert, NaN first, so that it shows in the weights;
// -inf is never chosen.  Values are compared as unsigned numbers of the same order;
// 16-bit ones share a word with the expert's complement, so that one warp
// reduction gives the largest and settles ties.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"
#include "rgg_rows.cuh"

namespace rgg {

constexpr int kRouteThreads = 256;
constexpr int kRouteMaxExperts = 4096;
constexpr int kRouteMaxChoices = 32;  // a lane each
constexpr float kRouteEps = 1e-20f;

template <typename T>
struct RouteKey;  // order(x): the value's place in the order, unsigned; kNegInf: that of -inf, below all others

template <>
struct RouteKey<float> {
    static constexpr bool kPacked = false;
    static constexpr uint32_t kNegInf = 0x007fffffu;
    static __device__ __forceinline__ uint32_t order(float x) {
        const uint32_t b = __float_as_uint(x + 0.0f);  // -0 as 0
        return x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    }
    static __device__ __forceinline__ float value(uint32_t o) {
        return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
    }
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float from_float(float x) { return x; }
};

// 16-bit values with the sign in the top bit; bits of a value and its place in the order.
__device__ __forceinline__ uint32_t order16(uint32_t b) {
    return b == 0x8000u ? 0x8000u : (b & 0x8000u) ? (~b & 0xffffu) : (b | 0x8000u);  // -0 as 0
}
__device__ __forceinline__ uint16_t bits16(uint32_t o) {
    return static_cast<uint16_t>((o & 0x8000u) ? o & 0x7fffu : ~o);
}

template <>
struct RouteKey<__nv_bfloat16> {
    static constexpr bool kPacked = true;
    static constexpr uint32_t kNegInf = 0x007fu;
    static __device__ __forceinline__ uint32_t order(__nv_bfloat16 x) {
        return __hisnan(x) ? 0xffffu : order16(__bfloat16_as_ushort(x));
    }
    static __device__ __forceinline__ float value(uint32_t o) { return __bfloat162float(__ushort_as_bfloat16(bits16(o))); }
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};

template <>
struct RouteKey<__half> {
    static constexpr bool kPacked = true;
    static constexpr uint32_t kNegInf = 0x03ffu;
    static __device__ __forceinline__ uint32_t order(__half x) {
        return __hisnan(x) ? 0xffffu : order16(__half_as_ushort(x));
    }
    static __device__ __forceinline__ float value(uint32_t o) { return __half2float(__ushort_as_half(bits16(o))); }
    static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.0f / (1.0f + expf(-x)); }
// A softmax's sum to divide by: rows without a choice hold zeros only; NaN stays.
__device__ __forceinline__ float not_zero(float total) { return total == 0.0f ? 1.0f : total; }

// V: logits a lane, E <= 32 V.
template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int k,
                                                              int flags, float scale, int32_t* __restrict__ experts,
                                                              float* __restrict__ weights) {
    using Key = RouteKey<T>;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool sigmoid = flags & RGG_ROUTE_SIGMOID, renormalize = flags & RGG_ROUTE_RENORMALIZE;
    for (RowItems it(tokens, 1); it.left(); it.next()) {
        const T* row = logits + it.item * E;
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = 32 * i + lane;
            uint32_t o = 0;  // below every logit
            if (e < E) {
                o = Key::order(row[e]);
                if constexpr (Key::kPacked) o = (o << 16) | (0xffffu - e);
            }
            key[i] = o;
        }
        auto best = [&]() {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) m = max(m, key[i]);
            return m;
        };
        uint32_t m = best();
        float top = 0.0f, total = 0.0f;
        if (!sigmoid && !renormalize) {
            const uint32_t first = __reduce_max_sync(0xffffffffu, m);
            top = Key::value(Key::kPacked ? first >> 16 : first);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t o = Key::kPacked ? key[i] >> 16 : key[i];
                if (o > Key::kNegInf) total += expf(Key::value(o) - top);
            }
            total = warp_sum(total);
        }
        uint32_t mine = 0;  // order of this lane's choice
        int32_t expert = -1;
        for (int j = 0; j < k; ++j) {
            const uint32_t M = __reduce_max_sync(0xffffffffu, m);
            if ((Key::kPacked ? M >> 16 : M) <= Key::kNegInf) break;
            if constexpr (Key::kPacked) {
                if (lane == j) {
                    mine = M >> 16;
                    expert = static_cast<int32_t>(0xffffu - (M & 0xffffu));
                }
                if (m == M) {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = key[i] == M ? 0u : key[i];
                    m = best();
                }
            } else {
                uint32_t e = 0xffffffffu;  // the lane's lowest expert of that value
                if (m == M) {
#pragma unroll
                    for (int i = V - 1; i >= 0; --i)
                        if (key[i] == M) e = 32 * i + lane;
                }
                const uint32_t first = __reduce_min_sync(0xffffffffu, e);
                if (lane == j) {
                    mine = M;
                    expert = static_cast<int32_t>(first);
                }
                if (e == first) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (static_cast<uint32_t>(32 * i + lane) == first) key[i] = 0u;
                    m = best();
                }
            }
        }
        float w = 0.0f;
        const float l = Key::value(mine);
        if (sigmoid) {
            if (expert >= 0) w = sigmoid_f32(l);
            if (renormalize) w = w / (warp_sum(w) + kRouteEps);
        } else if (renormalize) {
            top = __shfl_sync(0xffffffffu, l, 0);
            if (expert >= 0) w = expf(l - top);
            w = w / not_zero(warp_sum(w));
        } else if (expert >= 0) {
            w = expf(l - top) / total;
        }
        if (lane < k) {
            experts[it.item * k + lane] = expert;
            weights[it.item * k + lane] = w * scale;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kRouteThreads)
    route_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ experts,
                          const float* __restrict__ dweights, int64_t tokens, int E, int k, int flags, float scale,
                          int wide, T* __restrict__ dlogits, int32_t* status) {
    using Key = RouteKey<T>;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool sigmoid = flags & RGG_ROUTE_SIGMOID, renormalize = flags & RGG_ROUTE_RENORMALIZE;
    for (RowItems it(tokens, 1); it.left(); it.next()) {
        const T* row = logits + it.item * E;
        T* out = dlogits + it.item * E;
        int32_t e = -1;
        float g = 0.0f, l = 0.0f;
        if (lane < k) {
            e = checked_row(experts[it.item * k + lane], E, status);
            if (e >= 0) {
                g = dweights[it.item * k + lane] * scale;
                l = Key::to_float(row[e]);
            }
        }
        const bool chosen = e >= 0;
        float d = 0.0f;
        if (!sigmoid && !renormalize) {
            float top = -INFINITY, total = 0.0f;
            for (int i = lane; i < E; i += 32) top = fmaxf(top, Key::to_float(row[i]));
            top = warp_max(top);
            if (top == -INFINITY) top = 0.0f;  // all masked: every weight is 0
            for (int i = lane; i < E; i += 32) total += expf(Key::to_float(row[i]) - top);
            total = not_zero(warp_sum(total));
            const float s = chosen ? expf(l - top) / total : 0.0f;
            const float sum = warp_sum(chosen ? g * s : 0.0f);
            for (int i = lane; i < E; i += 32)
                out[i] = Key::from_float(-sum * (expf(Key::to_float(row[i]) - top) / total));
            // an expert chosen twice has both gradients; its value is then written by each of its lanes alike
            float all = 0.0f;
            for (int j = 0; j < k; ++j) {
                const int32_t oe = __shfl_sync(0xffffffffu, e, j);
                const float og = __shfl_sync(0xffffffffu, g, j);
                if (oe == e) all += og;
            }
            d = s * (all - sum);
        } else {
            if (sigmoid) {
                const float s = chosen ? sigmoid_f32(l) : 0.0f;
                if (renormalize) {
                    const float total = warp_sum(s) + kRouteEps;
                    const float sum = warp_sum(chosen ? g * (s / total) : 0.0f);
                    d = chosen ? (g - sum) / total * s * (1.0f - s) : 0.0f;
                } else {
                    d = chosen ? g * s * (1.0f - s) : 0.0f;
                }
            } else {
                float top = warp_max(chosen ? l : -INFINITY);
                if (top == -INFINITY) top = 0.0f;
                float w = chosen ? expf(l - top) : 0.0f;
                w = w / not_zero(warp_sum(w));
                const float sum = warp_sum(chosen ? g * w : 0.0f);
                d = chosen ? w * (g - sum) : 0.0f;
            }
            if (wide) {  // rows of whole 16 bytes
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int i = lane; i < wide; i += 32) reinterpret_cast<uint4*>(out)[i] = zero;
            } else {
                for (int i = lane; i < E; i += 32) out[i] = Key::from_float(0.0f);
            }
            float all = 0.0f;
            for (int j = 0; j < k; ++j) {
                const int32_t oe = __shfl_sync(0xffffffffu, e, j);
                const float od = __shfl_sync(0xffffffffu, d, j);
                if (oe == e) all += od;
            }
            d = all;
        }
        __syncwarp();  // the row's other values are written before the choices'
        if (chosen) out[e] = Key::from_float(d);
    }
}

template <typename T, int V>
static cudaError_t launch_route(const void* logits, int64_t tokens, int E, int k, int flags, float scale,
                                int32_t* experts, float* weights, cudaStream_t st) {
    return launch_chained(route_kernel<T, V>, row_grid(tokens, kRouteThreads), kRouteThreads, 0, st,
                          static_cast<const T*>(logits), tokens, E, k, flags, scale, experts, weights);
}

template <typename T>
static cudaError_t launch_route_for(int E, const void* logits, int64_t tokens, int k, int flags, float scale,
                                    int32_t* experts, float* weights, cudaStream_t st) {
    if (E <= 32) return launch_route<T, 1>(logits, tokens, E, k, flags, scale, experts, weights, st);
    if (E <= 64) return launch_route<T, 2>(logits, tokens, E, k, flags, scale, experts, weights, st);
    if (E <= 128) return launch_route<T, 4>(logits, tokens, E, k, flags, scale, experts, weights, st);
    if (E <= 256) return launch_route<T, 8>(logits, tokens, E, k, flags, scale, experts, weights, st);
    if (E <= 512) return launch_route<T, 16>(logits, tokens, E, k, flags, scale, experts, weights, st);
    if (E <= 1024) return launch_route<T, 32>(logits, tokens, E, k, flags, scale, experts, weights, st);
    return launch_route<T, 128>(logits, tokens, E, k, flags, scale, experts, weights, st);
}

static rgg_status route_check(const rgg_handle* h, const void* logits, int dtype, int64_t T, int E, int k, int flags,
                              float scale) {
    if (!h || T < 0 || T >= (int64_t(1) << 31) || E < 1 || k < 1 || k > E || scale != scale) return RGG_ERR_INVALID_ARG;
    if (flags & ~(RGG_ROUTE_SIGMOID | RGG_ROUTE_RENORMALIZE)) return RGG_ERR_INVALID_ARG;
    if (dtype != RGG_BF16 && dtype != RGG_FP32 && dtype != RGG_FP16) return RGG_ERR_INVALID_ARG;
    if (E > kRouteMaxExperts || k > kRouteMaxChoices) return RGG_ERR_UNSUPPORTED;
    if (T > 0 && (!logits || !host_aligned(logits, dtype == RGG_FP32 ? 4 : 2))) return RGG_ERR_INVALID_ARG;
    return RGG_OK;
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_route_topk(rgg_handle* h, const void* logits, int dtype, int64_t T, int E, int k, int flags,
                                     float scale, int32_t* experts, float* weights, void* stream) {
    rgg_status s = route_check(h, logits, dtype, T, E, k, flags, scale);
    if (s != RGG_OK) return s;
    if (T == 0) return RGG_OK;
    if (!experts || !weights || !host_aligned(experts, 4) || !host_aligned(weights, 4)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err =
        dtype == RGG_FP32 ? launch_route_for<float>(E, logits, T, k, flags, scale, experts, weights, st)
        : dtype == RGG_BF16
            ? launch_route_for<__nv_bfloat16>(E, logits, T, k, flags, scale, experts, weights, st)
            : launch_route_for<__half>(E, logits, T, k, flags, scale, experts, weights, st);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "route_topk launch");
}

extern "C" rgg_status rgg_route_topk_backward(rgg_handle* h, const void* logits, int dtype, const int32_t* experts,
                                              const float* dweights, void* dlogits, int64_t T, int E, int k, int flags,
                                              float scale, void* stream) {
    rgg_status s = route_check(h, logits, dtype, T, E, k, flags, scale);
    if (s != RGG_OK) return s;
    if (T == 0) return RGG_OK;
    const int size = dtype == RGG_FP32 ? 4 : 2;
    if (!experts || !dweights || !dlogits || !host_aligned(experts, 4) || !host_aligned(dweights, 4) ||
        !host_aligned(dlogits, size))
        return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int wide = (E * size % 16 == 0 && host_aligned(dlogits, 16)) ? E * size / 16 : 0;
    const int grid = row_grid(T, kRouteThreads);
    cudaError_t err;
    if (dtype == RGG_FP32)
        err = launch_chained(route_backward_kernel<float>, grid, kRouteThreads, 0, st, static_cast<const float*>(logits),
                             experts, dweights, T, E, k, flags, scale, wide, static_cast<float*>(dlogits), dev.status);
    else if (dtype == RGG_BF16)
        err = launch_chained(route_backward_kernel<__nv_bfloat16>, grid, kRouteThreads, 0, st,
                             static_cast<const __nv_bfloat16*>(logits), experts, dweights, T, E, k, flags, scale, wide,
                             static_cast<__nv_bfloat16*>(dlogits), dev.status);
    else
        err = launch_chained(route_backward_kernel<__half>, grid, kRouteThreads, 0, st,
                             static_cast<const __half*>(logits), experts, dweights, T, E, k, flags, scale, wide,
                             static_cast<__half*>(dlogits), dev.status);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "route_topk_backward launch");
}
