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
// with w before the scale.  The differences are formed so that they keep their bits where a weight is nearly 1.
//
// A warp takes a token, each lane up to 8 logits (kWide: neighbouring ones, read by one or
// two 16-byte loads; else l, l + 32, ...; above 256 experts more).  The order is by value,
// ties to the lower expert, NaN first, so that it shows in the weights; -inf is
// never chosen.  Values are compared as unsigned numbers of the same order, joined with
// the expert's complement, which settles ties: 16-bit values share a 32-bit word with it.
// Each lane sorts its own by a network; then k times a warp reduction finds the largest of
// the lanes' first, and its lane moves on to its next.  Bound by the instructions that
// takes (83 % of the issue slots): 32,768 tokens x 256 experts, k = 8, bf16 (17 MB) 14.5 us, fp32
// 21; searching all logits of a lane k times took 24 and 30.  Tokens in turn on fewer blocks, the
// next one's logits on their way, were slower (16.4).  Above 256 experts a lane keeps its logits unsorted and
// searches them all again after each choice of its own; above 1,024 they no longer fit its registers
// (4,096 x 4,096, softmax over all, 63 us of 10; its gradient 33).  The gradient of 32,768 x 256 bf16, k = 8: 6.2
// to 6.6 us where the choices alone have one, 10.9 by softmax over all.
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

// A logit's place in the order: the bits of an fp32 number as an unsigned one.  Adding 0 makes 0 of -0, and of any NaN the
// positive one, which comes out on top.  16-bit values keep their bits in the upper half.
__device__ __forceinline__ uint32_t route_order(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float route_value(uint32_t order) {
    return __uint_as_float(order ^ ((order & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kRouteNegInf = 0x007fffffu;  // route_order(-inf): nothing above it is masked

template <typename T>
struct RouteType;
template <>
struct RouteType<float> {
    using Key = uint64_t;
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float from_float(float x) { return x; }
};
template <>
struct RouteType<__nv_bfloat16> {
    using Key = uint32_t;
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct RouteType<__half> {  // as fp32 (its 19 bits and an expert's 12 would fit a 32-bit key of their own: not built)
    using Key = uint64_t;
    static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
};

// Value and expert in one number: the larger value first, then the lower expert.  0 is below all of them.
template <typename Key>
__device__ __forceinline__ Key route_key(float x, uint32_t expert) {
    if constexpr (sizeof(Key) == 4) return (route_order(x) & 0xffff0000u) | (0xffffu - expert);
    else return (static_cast<uint64_t>(route_order(x)) << 32) | (0xffffu - expert);
}
template <typename Key>
__device__ __forceinline__ uint32_t key_order(Key key) {  // of bf16 -inf, too, this is kRouteNegInf or less
    if constexpr (sizeof(Key) == 4) return key & 0xffff0000u;
    else return static_cast<uint32_t>(key >> 32);
}
template <typename Key>
__device__ __forceinline__ float key_value(Key key) {
    uint32_t order = key_order(key);
    if (sizeof(Key) == 4 && !(order & 0x80000000u)) order |= 0xffffu;  // the lower half of a negative number's
    return route_value(order);
}
template <typename Key>
__device__ __forceinline__ int32_t key_expert(Key key) {
    return static_cast<int32_t>(0xffffu - static_cast<uint32_t>(key & 0xffffu));
}
// The largest of the warp's, in every lane.
__device__ __forceinline__ uint32_t warp_max_key(uint32_t key) { return __reduce_max_sync(0xffffffffu, key); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t key) {
    const uint32_t hi = static_cast<uint32_t>(key >> 32);
    const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
    return (static_cast<uint64_t>(top) << 32) | __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(key) : 0u);
}

template <typename Key>
__device__ __forceinline__ void order_pair(Key& a, Key& b) {
    const Key lo = a < b ? a : b;
    a = a < b ? b : a;
    b = lo;
}
// Largest first: odd-even merge networks for 2, 4 and 8.
template <typename Key, int V>
__device__ __forceinline__ void sort_lane(Key (&k)[V]) {
    static_assert(V <= 8, "");
    if constexpr (V >= 2)
#pragma unroll
        for (int i = 0; i < V; i += 2) order_pair(k[i], k[i + 1]);
    if constexpr (V >= 4)
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            order_pair(k[i], k[i + 2]);
            order_pair(k[i + 1], k[i + 3]);
            order_pair(k[i + 1], k[i + 2]);
        }
    if constexpr (V == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) order_pair(k[i], k[i + 4]);
        order_pair(k[2], k[4]);
        order_pair(k[3], k[5]);
        order_pair(k[1], k[2]);
        order_pair(k[3], k[4]);
        order_pair(k[5], k[6]);
    }
}

// A lane's logits of a row: kWide, V neighbouring ones in 16-byte loads (E = 32 V); else l, l + 32, ..., -inf past E.
template <typename T, int V, bool kWide>
struct RouteRow {
    static __device__ __forceinline__ int expert(int i, int lane) { return kWide ? V * lane + i : 32 * i + lane; }
    static __device__ __forceinline__ void load(const T* row, int E, int lane, float (&x)[V]) {
        if constexpr (kWide) {
            constexpr int kPer = 16 / sizeof(T);
            static_assert(V % kPer == 0, "");
#pragma unroll
            for (int i = 0; i < V; i += kPer) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + V * lane + i));
                const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
                for (int j = 0; j < kPer; ++j) x[i + j] = RouteType<T>::to_float(t[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = 32 * i + lane < E ? RouteType<T>::to_float(row[32 * i + lane]) : -INFINITY;
        }
    }
    static __device__ __forceinline__ void store(T* row, int E, int lane, const float (&x)[V]) {
        if constexpr (kWide) {
            constexpr int kPer = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < V; i += kPer) {
                uint4 w;
                T* t = reinterpret_cast<T*>(&w);
#pragma unroll
                for (int j = 0; j < kPer; ++j) t[j] = RouteType<T>::from_float(x[i + j]);
                *reinterpret_cast<uint4*>(row + V * lane + i) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (32 * i + lane < E) row[32 * i + lane] = RouteType<T>::from_float(x[i]);
        }
    }
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
template <typename T, int V, bool kWide>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int k,
                                                              int flags, float scale, int32_t* __restrict__ experts,
                                                              float* __restrict__ weights) {
    using Key = typename RouteType<T>::Key;
    using Row = RouteRow<T, V, kWide>;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool sigmoid = flags & RGG_ROUTE_SIGMOID, renormalize = flags & RGG_ROUTE_RENORMALIZE;
    for (RowItems it(tokens, 1); it.left(); it.next()) {
        float x[V];
        Row::load(logits + it.item * E, E, lane, x);
        Key key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = route_key<Key>(x[i], Row::expert(i, lane));
        Key head;  // the lane's largest that is left
        auto best = [&]() {
            head = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) head = key[i] > head ? key[i] : head;
        };
        if constexpr (V <= 8) {
            sort_lane<Key, V>(key);
            head = key[0];
        } else {
            best();
        }
        Key mine = 0;  // this lane's choice
        for (int j = 0; j < k; ++j) {
            const Key top = warp_max_key(head);
            if (key_order(top) <= kRouteNegInf) break;
            if (lane == j) mine = top;
            if (head == top) {
                if constexpr (V <= 8) {
#pragma unroll
                    for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
                    key[V - 1] = 0;
                    head = key[0];
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) key[i] = key[i] == top ? 0 : key[i];
                    best();
                }
            }
        }
        const bool chosen = mine != 0;
        const float l = key_value(mine);
        float w = 0.0f;
        if (sigmoid) {
            if (chosen) w = sigmoid_f32(l);
            if (renormalize) w = w / (warp_sum(w) + kRouteEps);
        } else {
            const float top = __shfl_sync(0xffffffffu, l, 0);
            if (chosen) w = expf(l - top);
            float total = w;
            if (!renormalize) {
                total = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) total += x[i] == -INFINITY ? 0.0f : expf(x[i] - top);
            }
            w = w / not_zero(warp_sum(total));
        }
        if (lane < k) {
            experts[it.item * k + lane] = chosen ? key_expert(mine) : -1;
            weights[it.item * k + lane] = chosen ? w * scale : 0.0f;
        }
    }
}

// Sums and maxima over groups of kLanes neighbouring lanes.
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// A choice as a lane of the backward pass has it: its gradient (times the scale) and its expert's logit; expert -1: none.
// kLanes lanes a token, the lane's place among them its choice.  A token that names an expert twice has both
// gradients: joined() gives each of its lanes their sum.
template <typename T, int kLanes>
struct RouteChoice {
    int32_t expert = -1;
    float g = 0.0f, l = 0.0f;
    uint32_t same;
    bool twice;
    int k;

    __device__ __forceinline__ RouteChoice(const T* row, const int32_t* experts, const float* dweights, bool in, int64_t token,
                                           int lane, int E, int k_, float scale, int32_t* status)
        : k(k_) {
        const int j = lane % kLanes;
        if (in && j < k) {
            expert = checked_row(experts[token * k + j], E, status);
            if (expert >= 0) {
                g = dweights[token * k + j] * scale;
                l = RouteType<T>::to_float(row[expert]);
            }
        }
        same = __match_any_sync(0xffffffffu, expert >= 0 ? expert * (32 / kLanes) + lane / kLanes : -1);
        twice = __any_sync(0xffffffffu, expert >= 0 && (same & (same - 1)) != 0);
    }
    __device__ __forceinline__ bool chosen() const { return expert >= 0; }
    __device__ __forceinline__ float joined(float v) const {
        if (!twice) return v;
        float all = 0.0f;
        const int first = (threadIdx.x & 31) / kLanes * kLanes;
        for (int j = 0; j < k; ++j) {
            const float other = __shfl_sync(0xffffffffu, v, first + j);
            if (same >> (first + j) & 1u) all += other;
        }
        return all;
    }
};

// The gradient by a row's logits for softmax over all experts, which reads the whole row: a warp a token, V logits a lane.
template <typename T, int V, bool kWide>
__global__ void __launch_bounds__(kRouteThreads)
    route_backward_dense_kernel(const T* __restrict__ logits, const int32_t* __restrict__ experts,
                                const float* __restrict__ dweights, int64_t tokens, int E, int k, float scale,
                                T* __restrict__ dlogits, int32_t* status) {
    using Row = RouteRow<T, V, kWide>;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (RowItems it(tokens, 1); it.left(); it.next()) {
        const T* row = logits + it.item * E;
        T* out = dlogits + it.item * E;
        float x[V];
        Row::load(row, E, lane, x);
        const RouteChoice<T, 32> c(row, experts, dweights, true, it.item, lane, E, k, scale, status);
        float top = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
        top = warp_max(top);
        if (top == -INFINITY) top = 0.0f;  // all masked: every weight is 0
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = expf(x[i] - top);
            total += x[i];
        }
        const float inverse = 1.0f / not_zero(warp_sum(total));
        const float s = c.chosen() ? expf(c.l - top) * inverse : 0.0f, g = c.joined(c.g);
        const float sum = warp_sum(c.g * s);
        float d = s * (g - sum);
        const uint32_t tops = inverse > 0.5f ? __ballot_sync(0xffffffffu, c.chosen() && c.l == top) : 0u;
        if (tops) {
            // A choice t with more than half of the weight, whose gradient g - sum would leave few bits: as differences
            // from it, (g - g_t) - (sum over the other choices of g s - g_t (1 - s_t)), 1 - s_t from the others.
            const int32_t t = __shfl_sync(0xffffffffu, c.expert, __ffs(tops) - 1);
            const float g_t = __shfl_sync(0xffffffffu, g, __ffs(tops) - 1);
            float others = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) others += Row::expert(i, lane) == t ? 0.0f : x[i];
            const float rest = warp_sum(c.expert == t ? 0.0f : c.g * s);
            d = s * ((g - g_t) - (rest - g_t * (warp_sum(others) * inverse)));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= -sum * inverse;
        Row::store(out, E, lane, x);
        __syncwarp();  // the row's other values are written before the choices'
        if (c.chosen()) out[c.expert] = RouteType<T>::from_float(d);
    }
}

// For the other rules, which have a gradient at the choices alone: zeros, and the choices' values behind them.  As many
// tokens a warp as it has lanes for their choices (32,768 tokens x 256, k = 8: a token a warp 9.3 us).
template <typename T, int kLanes>
__global__ void __launch_bounds__(kRouteThreads)
    route_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ experts,
                          const float* __restrict__ dweights, int64_t tokens, int E, int k, int flags, float scale,
                          int wide, T* __restrict__ dlogits, int32_t* status) {
    constexpr int kTokens = 32 / kLanes;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool sigmoid = flags & RGG_ROUTE_SIGMOID, renormalize = flags & RGG_ROUTE_RENORMALIZE;
    for (RowItems it((tokens + kTokens - 1) / kTokens, 1); it.left(); it.next()) {
        const int64_t t = it.item * kTokens + lane / kLanes;
        const bool in = t < tokens;
        T* out = dlogits + t * E;
        if (in) {
            const int j = lane % kLanes;
            if (wide) {  // rows of whole 16 bytes
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                for (int i = j; i < wide; i += kLanes) reinterpret_cast<uint4*>(out)[i] = zero;
            } else {
                for (int i = j; i < E; i += kLanes) out[i] = RouteType<T>::from_float(0.0f);
            }
        }
        const RouteChoice<T, kLanes> c(logits + t * E, experts, dweights, in, t, lane, E, k, scale, status);
        // s and 1 - s from one exponential: from s, which is 1 in fp32 above a logit of 17, 1 - s would have few bits or none
        const float e = expf(-fabsf(c.l)), r = sigmoid && c.chosen() ? 1.0f / (1.0f + e) : 0.0f;
        const float s = c.l < 0.0f ? e * r : r, rest = c.l < 0.0f ? r : e * r;
        float d = c.g * s * rest;
        if (renormalize) {
            // g_i - sum g_j w_j as differences from the gradient g0 of the largest weight, (g_i - g0) - sum w_j (g_j - g0),
            // + g0 (1 - sum w_j): beside a weight of nearly 1 its own gradient would leave nothing of the others'
            const float top = group_max<kLanes>(c.chosen() ? c.l : -INFINITY);
            const int base = lane & ~(kLanes - 1);
            const uint32_t tops = __ballot_sync(0xffffffffu, c.chosen() && c.l == top) & (0xffffffffu >> (32 - kLanes) << base);
            const int largest = tops ? __ffs(tops) - 1 : base;
            const float g0 = __shfl_sync(0xffffffffu, c.g, largest);
            if (sigmoid) {
                const float inverse = 1.0f / (group_sum<kLanes>(s) + kRouteEps), w = s * inverse, diff = c.g - g0;
                d = (diff - group_sum<kLanes>(diff * w) + g0 * (kRouteEps * inverse)) * w * rest;
            } else {
                float w = c.chosen() ? expf(c.l - (top == -INFINITY ? 0.0f : top)) : 0.0f;
                w = w / not_zero(group_sum<kLanes>(w));
                d = w * ((c.g - g0) - group_sum<kLanes>((c.g - g0) * w));
            }
        }
        d = c.joined(c.chosen() ? d : 0.0f);
        __syncwarp();  // the zeros are written before the choices' values
        if (c.chosen()) out[c.expert] = RouteType<T>::from_float(d);
    }
}

struct RouteCall {
    const void* logits;
    int64_t T;
    int E, k, flags;
    float scale;
    int32_t* experts;  // the backward pass reads them
    float* weights;
    const float* dweights;
    void* dlogits;
    int32_t* status;
    cudaStream_t st;
};

template <typename T, int V, bool kWide>
static cudaError_t launch_route(const RouteCall& c) {
    const int grid = row_grid(c.T, kRouteThreads);
    if (!c.dlogits)
        return launch_chained(route_kernel<T, V, kWide>, grid, kRouteThreads, 0, c.st, static_cast<const T*>(c.logits), c.T,
                              c.E, c.k, c.flags, c.scale, c.experts, c.weights);
    return launch_chained(route_backward_dense_kernel<T, V, kWide>, grid, kRouteThreads, 0, c.st,
                          static_cast<const T*>(c.logits), static_cast<const int32_t*>(c.experts), c.dweights, c.T, c.E,
                          c.k, c.scale, static_cast<T*>(c.dlogits), c.status);
}

template <typename T>
static cudaError_t launch_route_for(const RouteCall& c) {
    constexpr int kPer = 16 / sizeof(T);
    const bool aligned = host_aligned(c.logits, 16) && host_aligned(c.dlogits, 16);
    if (c.dlogits && (c.flags & (RGG_ROUTE_SIGMOID | RGG_ROUTE_RENORMALIZE))) {
        const int wide = (c.E % kPer == 0 && host_aligned(c.dlogits, 16)) ? c.E / kPer : 0;
        const int tokens = c.k <= 8 ? 4 : c.k <= 16 ? 2 : 1;  // a warp
        auto kernel = tokens == 4 ? route_backward_kernel<T, 8> : tokens == 2 ? route_backward_kernel<T, 16>
                                                                              : route_backward_kernel<T, 32>;
        return launch_chained(kernel, row_grid((c.T + tokens - 1) / tokens, kRouteThreads), kRouteThreads, 0, c.st,
                              static_cast<const T*>(c.logits), static_cast<const int32_t*>(c.experts), c.dweights, c.T,
                              c.E, c.k, c.flags, c.scale, wide, static_cast<T*>(c.dlogits), c.status);
    }
    // Wide loads: lanes of whole 16-byte blocks, E = 32 V, among the V that a network sorts and that are whole blocks of
    // the type (bf16 8, fp32 4 and 8).  At 160, 192 or 224 experts a lane's part is none; above 256 the choices take the
    // time, not the loads.
    if (aligned && c.E == 256) return launch_route<T, 8, true>(c);
    if constexpr (kPer == 4) {
        if (aligned && c.E == 128) return launch_route<T, 4, true>(c);
    }
    if (c.E <= 32) return launch_route<T, 1, false>(c);
    if (c.E <= 64) return launch_route<T, 2, false>(c);
    if (c.E <= 128) return launch_route<T, 4, false>(c);
    if (c.E <= 256) return launch_route<T, 8, false>(c);
    if (c.E <= 512) return launch_route<T, 16, false>(c);
    if (c.E <= 1024) return launch_route<T, 32, false>(c);
    return launch_route<T, 128, false>(c);
}

static rgg_status route_run(int dtype, const RouteCall& c, const char* what) {
    cudaError_t err = dtype == RGG_FP32   ? launch_route_for<float>(c)
                      : dtype == RGG_BF16 ? launch_route_for<__nv_bfloat16>(c)
                                          : launch_route_for<__half>(c);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, what);
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
    const RouteCall c = {logits,  T,       E,       k,          flags,
                         scale,   experts, weights, nullptr,    nullptr,
                         nullptr, static_cast<cudaStream_t>(stream)};
    return route_run(dtype, c, "route_topk launch");
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
    const RouteCall c = {logits,
                         T,
                         E,
                         k,
                         flags,
                         scale,
                         const_cast<int32_t*>(experts),
                         nullptr,
                         dweights,
                         dlogits,
                         dev.status,
                         static_cast<cudaStream_t>(stream)};
    return route_run(dtype, c, "route_topk_backward launch");
}
