// rgg_grouped_gemm_wgrad: argument checks, tensor maps and the launch of the
// weight-gradient kernel (rgg_wgrad.cuh).
#include "rgg_wgrad.cuh"

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

// The multiplier and shift of wgrad_divide.
static void wgrad_divisor(int32_t d, uint32_t* by, int32_t* shift) {
    int32_t bits = 0;
    while ((int64_t(1) << bits) < d) ++bits;
    *shift = 30 + bits;
    *by = static_cast<uint32_t>((uint64_t(1) << *shift) / static_cast<uint64_t>(d) + 1);
}

struct WgradMaps {
    CUtensorMap x, x16, dy, dy16, dw;  // with boxes of 64 and of 16 rows
};

template <int BN, bool kF32, bool kAdd>
static cudaError_t launch_wgrad(int grid, size_t smem, cudaStream_t stream, const WgradMaps& m,
                                const WgradArgs& args) {
    auto kernel = grouped_wgrad_kernel<BN, kF32, kAdd>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_chained(kernel, grid, kWgradThreads, smem, stream, m.x, m.x16, m.dy, m.dy16, m.dw, args);
}

template <int BN>
static cudaError_t launch_wgrad_kind(int flags, int grid, size_t smem, cudaStream_t stream, const WgradMaps& m,
                                     const WgradArgs& args) {
    switch (flags) {
        case 0: return launch_wgrad<BN, false, false>(grid, smem, stream, m, args);
        case RGG_WGRAD_FP32: return launch_wgrad<BN, true, false>(grid, smem, stream, m, args);
        case RGG_WGRAD_ACCUMULATE: return launch_wgrad<BN, false, true>(grid, smem, stream, m, args);
        default: return launch_wgrad<BN, true, true>(grid, smem, stream, m, args);
    }
}

// dW[e] = (dW[e] +) the sum over the parts of expert e, in order, eight values a
// thread: bf16 results are rounded once, from the fp32 sum of everything.  Like
// the tiles' kernel it writes nothing where the offsets are not valid (there
// are then no parts either), and with accumulation leaves experts without rows alone.
template <bool kF32, bool kAdd>
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(const float4* __restrict__ parts, void* __restrict__ dW, const int32_t* __restrict__ offsets, int E,
                      int64_t M_tot, int64_t per_expert, int split) {
    extern __shared__ int32_t s_off[];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    if (!load_and_check_offsets(offsets, s_off, E, M_tot)) return;
    const int64_t total = per_expert * E;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        // i counts eighths of an expert's weight: per_expert of them
        const int64_t e = i / per_expert, at = i - e * per_expert;
        if (kAdd && s_off[e + 1] == s_off[e]) continue;
        const float4* p = parts + 2 * (e * split * per_expert + at);
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
        for (int s = 0; s < split; ++s, p += 2 * per_expert) {
            const float4 x = __ldg(p), y = __ldg(p + 1);
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
            b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
        }
        if constexpr (kF32) {
            float4* out = static_cast<float4*>(dW) + 2 * i;
            if constexpr (kAdd) {
                const float4 x = out[0], y = out[1];
                a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
                b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
            }
            out[0] = a;
            out[1] = b;
        } else {
            uint4* out = static_cast<uint4*>(dW) + i;
            if constexpr (kAdd) {
                const uint4 o = *out;
                a.x += __uint_as_float(o.x << 16); a.y += __uint_as_float(o.x & 0xffff0000u);
                a.z += __uint_as_float(o.y << 16); a.w += __uint_as_float(o.y & 0xffff0000u);
                b.x += __uint_as_float(o.z << 16); b.y += __uint_as_float(o.z & 0xffff0000u);
                b.z += __uint_as_float(o.w << 16); b.w += __uint_as_float(o.w & 0xffff0000u);
            }
            auto pack = [](float lo, float hi) { return pack_bf16x2(__float_as_uint(lo), __float_as_uint(hi)); };
            *out = make_uint4(pack(a.x, a.y), pack(a.z, a.w), pack(b.x, b.y), pack(b.z, b.w));
        }
    }
}

static cudaError_t launch_wgrad_join(int flags, int num_sms, const void* parts, void* dW, const int32_t* offsets, int E,
                                     int64_t M_tot, int64_t per_expert, int split, cudaStream_t stream) {
    const int64_t total = per_expert * E;
    const int grid = static_cast<int>(std::min<int64_t>((total + 255) / 256, 8LL * num_sms));
    auto kernel = flags == 0                          ? wgrad_join_kernel<false, false>
                  : flags == RGG_WGRAD_FP32           ? wgrad_join_kernel<true, false>
                  : flags == RGG_WGRAD_ACCUMULATE     ? wgrad_join_kernel<false, true>
                                                      : wgrad_join_kernel<true, true>;
    return launch_chained(kernel, grid, 256, 4u * static_cast<size_t>(E + 1), stream,
                          static_cast<const float4*>(parts), dW, offsets, E, M_tot, per_expert, split);
}

struct WgradShape {
    int bn, split;
};

// What the parts' sums take; for a split that wgrad_shape considers at most two tiles of 256 KB a pair.
static int64_t wgrad_parts_bytes(int split, int E, int K, int N) { return static_cast<int64_t>(split) * E * K * N * 4; }

constexpr int64_t kAnyRoom = INT64_MAX;

// The tile width and the parts an expert's rows are split into, by the time of
// the waves with the rows taken as even (us, fitted to this kernel: 0.30 a
// stage and 0.9 a tile of 256 columns, 0.6 of that for 128, over an expert's
// tiles in the mean), the sums' way through memory and the second launch.  The rows are split where the tiles are
// too few to fill the GPU: one expert of 16,384 rows, K = N = 1024 takes 37 us
// split and 48 unsplit, of 32,768 rows, K = N = 256, 23 and 76.  The parts take
// `room` bytes at most.
static WgradShape wgrad_shape(int pairs, int E, int64_t M_tot, int K, int N, bool f32, int want_bn, int64_t room) {
    WgradShape best = {want_bn ? want_bn : 256, 1};
    double least = 1e300;
    for (int bn : {256, 128}) {
        if (want_bn != 0 && bn != want_bn) continue;
        const int64_t tiles = static_cast<int64_t>(E) * ((K + kWgradBM - 1) / kWgradBM) * ((N + bn - 1) / bn);
        for (int split = 1; split <= 32; split *= 2) {
            const double stages = static_cast<double>(M_tot) / E / kWgradRows / split;
            if (split > 1 && (stages < 4.0 || tiles * split > 2 * pairs || wgrad_parts_bytes(split, E, K, N) > room))
                break;
            const double waves = static_cast<double>((tiles * split + pairs - 1) / pairs);
            // a last tile of up to 128 columns multiplies 128
            const int whole = N / bn, last = N % bn == 0 ? 0 : N % bn <= 128 ? 128 : bn;
            const double width = (whole * (bn + 64.0) + (last ? last + 64.0 : 0.0)) / (whole + (last ? 1 : 0)) / 320.0;
            double us = waves * (std::max(1.0, stages) * 0.30 + 0.9) * width;
            if (split > 1) {
                const double values = static_cast<double>(E) * K * N;
                us += 6.0 + values * (8.0 * split + (f32 ? 4.0 : 2.0)) / 4e6;  // parts written and read, at 4 TB/s
            }
            if (us < least) {
                least = us;
                best = {bn, split};
            }
        }
    }
    return best;
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_grouped_gemm_wgrad(rgg_handle* h, const void* X, const void* dY,
                                             const int32_t* group_offsets, void* dW, int E, int64_t M_tot, int K,
                                             int N, int flags, void* stream, const rgg_options* opt) {
    if (!h || !group_offsets || !dW) return RGG_ERR_INVALID_ARG;
    if ((flags & ~(RGG_WGRAD_FP32 | RGG_WGRAD_ACCUMULATE)) != 0) return RGG_ERR_INVALID_ARG;
    rgg_status s = host_check_sizes(E, M_tot, K, N);
    if (s != RGG_OK) return s;
    if (M_tot > 0 && (!X || !dY)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(dW, 16) || !host_aligned(group_offsets, 4) || !host_aligned(X, 16) || !host_aligned(dY, 16))
        return RGG_ERR_INVALID_ARG;
    const int want_bn = opt ? opt->bn : 0, want_stages = opt ? opt->stages : 0, max_ctas = opt ? opt->max_ctas : 0;
    if (opt && opt->bm != 0 && opt->bm != kWgradBM) return RGG_ERR_INVALID_ARG;
    if (want_bn != 0 && want_bn != 128 && want_bn != 256) return RGG_ERR_INVALID_ARG;
    if (want_stages != 0 && (want_stages < 2 || want_stages > kMaxStages)) return RGG_ERR_INVALID_ARG;
    if (max_ctas < 0 || max_ctas == 1) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");

    const int pairs = (max_ctas > 0 ? std::min(max_ctas, dev.num_sms) : dev.num_sms) / 2;
    auto tiles = [&](int bn) {
        return static_cast<int64_t>(E) * ((K + kWgradBM - 1) / kWgradBM) * ((N + bn - 1) / bn);
    };
    // A workspace of the size that the query gives is enough whatever the
    // options are: the rows are split into as many parts as fit it.
    const bool f32 = (flags & RGG_WGRAD_FP32) != 0;
    const int64_t room_bytes = opt && opt->workspace ? opt->workspace_bytes : 0;
    const WgradShape shape = wgrad_shape(pairs, E, M_tot, K, N, f32, want_bn, room_bytes);
    const int bn = shape.bn, split = shape.split;
    if (split > 1 && !host_aligned(opt->workspace, 16)) return RGG_ERR_INVALID_ARG;
    if (opt && opt->workspace && room_bytes < rgg_grouped_gemm_wgrad_workspace(h, E, M_tot, K, N, flags)) {
        const int wanted = wgrad_shape(pairs, E, M_tot, K, N, f32, want_bn, kAnyRoom).split;
        if (wanted > 1 && room_bytes < wgrad_parts_bytes(wanted, E, K, N)) return RGG_ERR_INVALID_ARG;
    }
    // where the tiles' sums go: dW, or each part's place in the workspace
    void* out = split > 1 ? opt->workspace : dW;
    const int out_flags = split > 1 ? RGG_WGRAD_FP32 : flags;
    if (tiles(bn) * split >= (int64_t(1) << 30)) return RGG_ERR_UNSUPPORTED;
    const int64_t room = static_cast<int64_t>(dev.smem_optin) - 1024 - wgrad_smem(bn, 0, E).total;
    const int per_stage = (2 + bn / 128) * static_cast<int>(kWgradPanel) + 8 * (3 + kWgradTailWarps);
    const int fit = static_cast<int>(std::min<int64_t>(8, room / per_stage));
    const int stages = want_stages ? want_stages : fit;
    if (stages < 2 || stages > fit) return RGG_ERR_UNSUPPORTED;
    // more than half of the SM's shared memory, so that one CTA lives on each SM
    const int smem = std::max<int>(static_cast<int>(wgrad_smem(bn, stages, E).total) + 1024,
                                   dev.smem_optin / 2 + 1024);

    // Without rows no copy is issued; the maps then stand on dW's memory.
    WgradMaps m;
    const int64_t rows = M_tot > 0 ? M_tot : 1;
    const void* px = M_tot > 0 ? X : dW;
    const void* py = M_tot > 0 ? dY : dW;
    s = host_encode_rows(px, rows, K, kWgradRows, &m.x);
    if (s == RGG_OK) s = host_encode_rows(px, rows, K, 16, &m.x16);
    if (s == RGG_OK) s = host_encode_rows(py, rows, N, kWgradRows, &m.dy);
    if (s == RGG_OK) s = host_encode_rows(py, rows, N, 16, &m.dy16);
    if (s == RGG_OK) s = host_encode_out(out, E * split, K, N, (out_flags & RGG_WGRAD_FP32) != 0, 32, &m.dw);
    if (s != RGG_OK) return s;

    WgradArgs a;
    a.offsets = group_offsets;
    a.X = static_cast<const __nv_bfloat16*>(X);
    a.dY = static_cast<const __nv_bfloat16*>(dY);
    a.dW = out;
    a.status = dev.status;
    a.M_tot = M_tot;
    a.E = E;
    a.K = K;
    a.N = N;
    a.split = split;
    a.tiles_n = (N + bn - 1) / bn;
    a.tiles_e = a.tiles_n * ((K + kWgradBM - 1) / kWgradBM);
    wgrad_divisor(a.tiles_n, &a.by_tiles_n, &a.shift_n);
    wgrad_divisor(a.tiles_e, &a.by_tiles_e, &a.shift_e);
    a.stages = stages;
    a.debug_flags = opt ? (opt->debug_flags & RGG_DEBUG_PRODUCER_STALL) : 0;
    a.timeout_ns = (opt && opt->timeout_ns) ? opt->timeout_ns : kHostDefaultTimeoutNs;
    const int grid = 2 * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(pairs, tiles(bn) * split)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = bn == 256 ? launch_wgrad_kind<256>(out_flags, grid, smem, st, m, a)
                                : launch_wgrad_kind<128>(out_flags, grid, smem, st, m, a);
    if (err == cudaSuccess && split > 1)
        err = launch_wgrad_join(flags, dev.num_sms, out, dW, group_offsets, E, M_tot,
                                static_cast<int64_t>(K) * N / 8, split, st);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "grouped_gemm_wgrad launch");
}

extern "C" int64_t rgg_grouped_gemm_wgrad_workspace(rgg_handle* h, int E, int64_t M_tot, int K, int N, int flags) {
    if (!h || host_check_sizes(E, M_tot, K, N) != RGG_OK) return 0;
    const WgradShape shape = wgrad_shape(std::max(1, host_device(h).num_sms / 2), E, M_tot, K, N,
                                         (flags & RGG_WGRAD_FP32) != 0, 0, kAnyRoom);
    return shape.split > 1 ? wgrad_parts_bytes(shape.split, E, K, N) : 0;
}
