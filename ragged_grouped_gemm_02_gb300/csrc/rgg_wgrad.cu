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
    // The narrower tile only where it fills more of the GPU in as many waves:
    // a wave costs the tile's columns and a fixed part, as in the forward plan.
    int bn = want_bn;
    if (bn == 0) {
        auto cost = [&](int b) { return (tiles(b) + pairs - 1) / pairs * (b + 64); };
        bn = cost(128) < cost(256) ? 128 : 256;
    }
    if (tiles(bn) >= (int64_t(1) << 30)) return RGG_ERR_UNSUPPORTED;
    const int64_t room = static_cast<int64_t>(dev.smem_optin) - 1024 - wgrad_smem(bn, 0, E).total;
    const int per_stage = (2 + bn / 128) * static_cast<int>(kWgradPanel) + 32;
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
    if (s == RGG_OK) s = host_encode_out(dW, E, K, N, (flags & RGG_WGRAD_FP32) != 0, 32, &m.dw);
    if (s != RGG_OK) return s;

    WgradArgs a;
    a.offsets = group_offsets;
    a.X = static_cast<const __nv_bfloat16*>(X);
    a.dY = static_cast<const __nv_bfloat16*>(dY);
    a.dW = dW;
    a.status = dev.status;
    a.M_tot = M_tot;
    a.E = E;
    a.K = K;
    a.N = N;
    a.tiles_n = (N + bn - 1) / bn;
    a.tiles_e = a.tiles_n * ((K + kWgradBM - 1) / kWgradBM);
    wgrad_divisor(a.tiles_n, &a.by_tiles_n, &a.shift_n);
    wgrad_divisor(a.tiles_e, &a.by_tiles_e, &a.shift_e);
    a.stages = stages;
    a.debug_flags = opt ? (opt->debug_flags & RGG_DEBUG_PRODUCER_STALL) : 0;
    a.timeout_ns = (opt && opt->timeout_ns) ? opt->timeout_ns : kHostDefaultTimeoutNs;
    const int grid = 2 * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(pairs, tiles(bn))));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = bn == 256 ? launch_wgrad_kind<256>(flags, grid, smem, st, m, a)
                                : launch_wgrad_kind<128>(flags, grid, smem, st, m, a);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "grouped_gemm_wgrad launch");
}
