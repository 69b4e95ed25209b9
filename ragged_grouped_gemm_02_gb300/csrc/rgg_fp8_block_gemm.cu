// rgg_grouped_gemm_fp8_block and rgg_grouped_gemm_swiglu_fp8_block: argument
// checks, tensor maps and the launch of the product with a scale per block of 128
// (rgg_fp8_block.cuh).
#include "rgg_fp8_block.cuh"

#include <algorithm>

#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

template <typename Kernel>
static cudaError_t launch_fp8_block(Kernel kernel, int grid, size_t smem, cudaStream_t stream, const FpMaps& maps,
                                    const FpArgs& args) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    // the kernel's warps share out the registers that it was launched with: other code than
    // was planned for would wait for ever
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess) return err;
    if (attr.numRegs != kFpRegsLaunch) return cudaErrorInvalidKernelImage;
    return launch_chained(kernel, grid, kFpThreads, smem, stream, maps, args);
}

static rgg_status fp8_block_call(rgg_handle* h, const void* x_codes, const float* x_scales, const void* w_codes,
                                 const float* w_scales, const int32_t* group_offsets, void* Y, float* h_scales, int E,
                                 int64_t M_tot, int K, int N, void* stream, const rgg_options* opt, bool gate_up) {
    if (!h || !group_offsets || !w_codes || !w_scales) return RGG_ERR_INVALID_ARG;
    rgg_status s = host_check_sizes(E, M_tot, K, N);
    if (s != RGG_OK) return s;
    if (K % 16 != 0 || (gate_up && (N % kFpBlock != 0 || N > kMaxWidth / 2))) return RGG_ERR_INVALID_ARG;
    if (M_tot > 0 && (!x_codes || !x_scales || !Y || (gate_up && !h_scales))) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(x_codes, 16) || !host_aligned(x_scales, 4) || !host_aligned(w_codes, 16) ||
        !host_aligned(w_scales, 4) || !host_aligned(Y, 16) || !host_aligned(h_scales, 4) ||
        !host_aligned(group_offsets, 4))
        return RGG_ERR_INVALID_ARG;
    const int want_bm = opt ? opt->bm : 0, want_stages = opt ? opt->stages : 0, max_ctas = opt ? opt->max_ctas : 0;
    if ((want_bm != 0 && want_bm != 128 && want_bm != 256) || max_ctas < 0) return RGG_ERR_INVALID_ARG;
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
    auto tile_n = [&](int bm) { return gate_up ? 128 : bm; };
    auto tiles_n = [&](int bm) { return (N + tile_n(bm) - 1) / tile_n(bm); };
    const int bm = want_bm ? want_bm : (avg > 128 && cap >= 2 ? 256 : 128);
    const bool pair = bm == 256;
    if (pair && cap < 2) return RGG_ERR_INVALID_ARG;
    const int64_t most = (M_tot / bm + E) * tiles_n(bm);
    if (most >= (int64_t(1) << 30)) return RGG_ERR_UNSUPPORTED;
    const uint32_t w_bytes = pair ? fp_w_bytes<true, false>() : gate_up ? fp_w_bytes<false, true>() : fp_w_bytes<false, false>();
    const int64_t fixed = fp_smem(0, E, w_bytes, gate_up).total;
    const int64_t per_stage = static_cast<int64_t>(kFpTile) + w_bytes + 16;
    const int64_t room = static_cast<int64_t>(dev.smem_optin) - 1024 - 16 - fixed;
    const int fit = static_cast<int>(std::min<int64_t>(kMaxStages, room / per_stage));
    const int stages = want_stages ? want_stages : fit;
    if (stages < 2 || stages > fit) return RGG_ERR_UNSUPPORTED;
    const int smem = std::max<int>(static_cast<int>(fp_smem(stages, E, w_bytes, gate_up).total) + 1024,
                                   dev.smem_optin / 2 + 1024);

    const int cols = gate_up ? 2 * N : N;
    FpMaps m;
    s = host_encode_codes(x_codes, M_tot, 1, K, 128, &m.x128);
    if (s == RGG_OK) s = host_encode_codes(x_codes, M_tot, 1, K, 32, &m.x32);
    if (s == RGG_OK) s = host_encode_codes(w_codes, cols, E, K, 128, &m.w128);
    if (s == RGG_OK) s = host_encode_codes(w_codes, cols, E, K, 64, &m.w64);
    if (s != RGG_OK) return s;

    FpArgs a = {};
    a.offsets = group_offsets;
    a.sx = x_scales;
    a.sw = w_scales;
    a.Y = gate_up ? nullptr : static_cast<__nv_bfloat16*>(Y);
    a.codes = gate_up ? static_cast<uint8_t*>(Y) : nullptr;
    a.scales = h_scales;
    a.status = dev.status;
    a.M_tot = M_tot;
    a.E = E;
    a.K = K;
    a.N = N;
    a.n_tiles_n = tiles_n(bm);
    a.stages = stages;
    a.y_vec32 = (N % 16 == 0 && host_aligned(Y, 32)) ? 1 : 0;
    a.n_major = avg >= 3 * bm ? 1 : 0;  // as the bf16 plan: the tiles that read one weight panel side by side
    a.debug_flags = opt ? (opt->debug_flags & RGG_DEBUG_PRODUCER_STALL) : 0;
    a.timeout_ns = (opt && opt->timeout_ns) ? opt->timeout_ns : kHostDefaultTimeoutNs;
    const int grid = static_cast<int>(pair ? 2 * std::max<int64_t>(1, std::min<int64_t>(cap / 2, most))
                                           : std::max<int64_t>(1, std::min<int64_t>(cap, most)));
    cudaError_t err =
        pair ? launch_fp8_block(gate_up ? grouped_fp8_block_pair_kernel<true> : grouped_fp8_block_pair_kernel<false>,
                                grid, smem, st, m, a)
             : launch_fp8_block(gate_up ? grouped_fp8_block_kernel<true> : grouped_fp8_block_kernel<false>, grid, smem,
                                st, m, a);
    return err == cudaSuccess ? RGG_OK : host_cuda_failure(err, "grouped_gemm_fp8_block launch");
}

}  // namespace rgg

using namespace rgg;

extern "C" rgg_status rgg_grouped_gemm_fp8_block(rgg_handle* h, const void* x_codes, const float* x_scales,
                                                 const void* w_codes, const float* w_scales,
                                                 const int32_t* group_offsets, void* Y, int E, int64_t M_tot, int K,
                                                 int N, void* stream, const rgg_options* opt) {
    return fp8_block_call(h, x_codes, x_scales, w_codes, w_scales, group_offsets, Y, nullptr, E, M_tot, K, N, stream, opt,
                          false);
}

extern "C" rgg_status rgg_grouped_gemm_swiglu_fp8_block(rgg_handle* h, const void* x_codes, const float* x_scales,
                                                        const void* w13_codes, const float* w13_scales,
                                                        const int32_t* group_offsets, void* h_codes, float* h_scales,
                                                        int E, int64_t M_tot, int K, int N, void* stream,
                                                        const rgg_options* opt) {
    return fp8_block_call(h, x_codes, x_scales, w13_codes, w13_scales, group_offsets, h_codes, h_scales, E, M_tot, K, N,
                          stream, opt, true);
}
