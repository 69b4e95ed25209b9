// rgg_grouped_gemm_mxfp4 and rgg_grouped_gemm_swiglu_mxfp4: argument checks,
// tensor maps and the launch of the MXFP4 product (rgg_mxfp4.cuh).
#include "rgg_mxfp4.cuh"

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

template <typename Kernel>
static cudaError_t launch_mxfp4(Kernel kernel, int grid, size_t smem, cudaStream_t stream, const MxMaps& maps,
                                const MxArgs& args) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_chained(kernel, grid, kMxThreads, smem, stream, maps, args);
}

static rgg_status mxfp4_call(rgg_handle* h, const void* x_codes, const void* x_scales, const void* w_codes,
                             const void* w_scales, const int32_t* group_offsets, void* Y, int E, int64_t M_tot, int K,
                             int N, void* stream, const rgg_options* opt, bool gate_up) {
    if (!h || !group_offsets || !w_codes || !w_scales) return RGG_ERR_INVALID_ARG;
    rgg_status s = host_check_sizes(E, M_tot, K, N);
    if (s != RGG_OK) return s;
    if (K % kMxBlock != 0 || (gate_up && (N % kMxRows != 0 || N > kMaxWidth / 2))) return RGG_ERR_INVALID_ARG;
    if (M_tot > 0 && (!x_codes || !x_scales || !Y)) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(x_codes, 16) || !host_aligned(x_scales, 16) || !host_aligned(w_codes, 16) ||
        !host_aligned(w_scales, 16) || !host_aligned(Y, 16) || !host_aligned(group_offsets, 4))
        return RGG_ERR_INVALID_ARG;
    const int want_bm = opt ? opt->bm : 0, want_stages = opt ? opt->stages : 0, max_ctas = opt ? opt->max_ctas : 0;
    if ((want_bm != 0 && want_bm != 128 && want_bm != 256) || max_ctas < 0)
        return RGG_ERR_INVALID_ARG;
    const int want_bn = opt ? opt->bn : 0;
    if (want_bn != 0 && want_bn != (want_bm == 0 ? want_bn : want_bm)) return RGG_ERR_INVALID_ARG;
    if (want_bn != 0 && want_bn != 128 && want_bn != 256) return RGG_ERR_INVALID_ARG;
    if (want_stages != 0 && (want_stages < 2 || want_stages > kMaxStages)) return RGG_ERR_INVALID_ARG;
    const HostDevice dev = host_device(h);
    HostDeviceScope scope(dev.device);
    if (scope.error() != cudaSuccess) return host_cuda_failure(scope.error(), "cudaSetDevice");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M_tot == 0) {
        cudaError_t err = launch_validate_offsets(group_offsets, E, M_tot, dev.status, st);
        return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "validate_offsets launch");
    }

    const int cap = max_ctas > 0 ? std::min(max_ctas, dev.num_sms) : dev.num_sms;
    const int64_t avg = (M_tot + E - 1) / E;
    auto tiles_n = [&](int b) { return (N + (gate_up ? b / 2 : b) - 1) / (gate_up ? b / 2 : b); };
    int b = want_bm ? want_bm : want_bn;
    if (b == 0) {
        // The shape with the shorter waves, experts taken as balanced: a tile
        // costs a fixed part and a part per stage of 256 of K, fitted in us to
        // 10 752 and 8 192 single tiles, 2 816 and 2 048 pair tiles of K = 1024
        // and 6144 (single 1.78 and 5.86, gate-up 7.2; pair 3.5 and 9.0).
        // Chosen by rows alone (pairs above 128), 64 experts x 256 rows of
        // K = 1024 took 48 us on pairs, 40 on single CTAs.
        const double kb = (K + kMxStageK - 1) / kMxStageK;
        auto waves = [&](int bb, int units) {
            const int64_t tiles = E * ((avg + bb - 1) / bb) * tiles_n(bb);
            return static_cast<double>((tiles + units - 1) / units);
        };
        const double single = waves(128, cap) * (0.96 + (gate_up ? 0.26 : 0.204) * kb);
        const double paired = cap >= 2 ? waves(256, cap / 2) * (2.4 + 0.275 * kb) : 1e300;
        b = (avg > 128 && paired < single) ? 256 : 128;
    }
    const bool pair = b == 256;
    if (pair && cap < 2) return RGG_ERR_INVALID_ARG;
    // blocks of scales are counted in 32 bits
    if (static_cast<int64_t>(E) * ((static_cast<int64_t>(gate_up ? 2 : 1) * N + kMxRows - 1) / kMxRows) >=
        (int64_t(1) << 31))
        return RGG_ERR_UNSUPPORTED;
    const int64_t most = (M_tot / b + E) * tiles_n(b);
    if (most >= (int64_t(1) << 30)) return RGG_ERR_UNSUPPORTED;
    const int64_t room = static_cast<int64_t>(dev.smem_optin) - 1024 - mx_smem(0, E).total;
    const int per_stage = static_cast<int>(mx_smem(1, E).total - mx_smem(0, E).total);
    const int fit = static_cast<int>(std::min<int64_t>(kMaxStages, room / per_stage));
    const int stages = want_stages ? want_stages : fit;
    if (stages < 2 || stages > fit) return RGG_ERR_UNSUPPORTED;
    const int smem = std::max<int>(static_cast<int>(mx_smem(stages, E).total) + 1024, dev.smem_optin / 2 + 1024);

    const int cols = gate_up ? 2 * N : N;
    const int64_t kblocks = mx_k_blocks(K);
    MxMaps m;
    s = host_encode_codes(x_codes, M_tot, 1, K / 2, 128, &m.x128);
    if (s == RGG_OK) s = host_encode_codes(x_codes, M_tot, 1, K / 2, 32, &m.x32);
    if (s == RGG_OK) s = host_encode_codes(w_codes, cols, E, K / 2, 128, &m.w128);
    if (s == RGG_OK) s = host_encode_codes(w_codes, cols, E, K / 2, 64, &m.w64);
    if (s == RGG_OK) s = host_encode_words(x_scales, mx_row_blocks(M_tot, E), kblocks * (kMxBlockBytes / 4), 256, &m.sx);
    if (s == RGG_OK)
        s = host_encode_words(w_scales, static_cast<int64_t>(E) * ((cols + kMxRows - 1) / kMxRows),
                              kblocks * (kMxBlockBytes / 4), 256, &m.sw);
    if (s != RGG_OK) return s;

    MxArgs a;
    a.offsets = group_offsets;
    a.Y = static_cast<__nv_bfloat16*>(Y);
    a.status = dev.status;
    a.M_tot = M_tot;
    a.E = E;
    a.K = K;
    a.N = N;
    a.n_tiles_n = tiles_n(b);
    a.stages = stages;
    a.y_vec32 = (N % 16 == 0 && host_aligned(Y, 32)) ? 1 : 0;
    a.n_major = avg >= 3 * b ? 1 : 0;  // as the bf16 plan: the tiles that read one weight panel side by side
    a.debug_flags = opt ? (opt->debug_flags & RGG_DEBUG_PRODUCER_STALL) : 0;
    a.timeout_ns = (opt && opt->timeout_ns) ? opt->timeout_ns : kHostDefaultTimeoutNs;
    const int grid = static_cast<int>(pair ? 2 * std::max<int64_t>(1, std::min<int64_t>(cap / 2, most))
                                           : std::max<int64_t>(1, std::min<int64_t>(cap, most)));
    cudaError_t err = pair ? launch_mxfp4(gate_up ? grouped_mxfp4_pair_kernel<true> : grouped_mxfp4_pair_kernel<false>,
                                          grid, smem, st, m, a)
                           : launch_mxfp4(gate_up ? grouped_mxfp4_kernel<true> : grouped_mxfp4_kernel<false>, grid,
                                          smem, st, m, a);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "grouped_gemm_mxfp4 launch");
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_grouped_gemm_mxfp4(rgg_handle* h, const void* x_codes, const void* x_scales,
                                             const void* w_codes, const void* w_scales,
                                             const int32_t* group_offsets, void* Y, int E, int64_t M_tot, int K,
                                             int N, void* stream, const rgg_options* opt) {
    return mxfp4_call(h, x_codes, x_scales, w_codes, w_scales, group_offsets, Y, E, M_tot, K, N, stream, opt, false);
}

extern "C" rgg_status rgg_grouped_gemm_swiglu_mxfp4(rgg_handle* h, const void* x_codes, const void* x_scales,
                                                    const void* w13_codes, const void* w13_scales,
                                                    const int32_t* group_offsets, void* H, int E, int64_t M_tot,
                                                    int K, int N, void* stream, const rgg_options* opt) {
    return mxfp4_call(h, x_codes, x_scales, w13_codes, w13_scales, group_offsets, H, E, M_tot, K, N, stream, opt, true);
}
