// rgg_grouped_gemm_fp8_block and rgg_grouped_gemm_swiglu_fp8_block: argument
// checks, tensor maps and the launch of the product with a scale per block of 128
// (rgg_fp8_block.cuh).
#include "rgg_fp8_block.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

using FpKernel = void (*)(FpMaps, FpArgs);
constexpr int kFpKernels = 5;  // of which `which` numbers one

// Once for each kernel and device: shared memory up to the device's most, and that its warps find the registers they share
// out (with other code than was planned for they would wait for ever).
static cudaError_t prepare_fp8_block(FpKernel kernel, int which, int regs, const HostDevice& dev) {
    static std::atomic<uint64_t> ready[kFpKernels];
    const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
    if (ready[which].load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.smem_optin);
    if (err != cudaSuccess) return err;
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, kernel);
    if (err != cudaSuccess) return err;
    if (attr.numRegs != regs) return cudaErrorInvalidKernelImage;
    ready[which].fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
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
    if (opt && opt->bn != 0 && opt->bn != 128 && opt->bn != 256) return RGG_ERR_INVALID_ARG;
    if (opt && opt->bn == 128 && (want_bm == 256 || gate_up)) return RGG_ERR_INVALID_ARG;
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
    const double avg = static_cast<double>(M_tot) / E;
    auto tile_n = [&](int shape) { return gate_up || shape == kFpNarrow ? 128 : 256; };
    auto tiles_n = [&](int shape) { return (N + tile_n(shape) - 1) / tile_n(shape); };
    const int want_bn = opt ? opt->bn : 0;
    const bool narrow_ok = !gate_up && want_bn != 256;
    int shape;
    if (want_bm == 256) {
        shape = kFpPair;
    } else if (want_bn == 128 && !gate_up) {
        shape = kFpNarrow;
    } else if (want_bn == 256 && want_bm == 128) {
        shape = kFpWide;
    } else if (avg <= 128) {
        // The weights' bytes bound the product, and more, smaller tiles keep all SMs reading (32 experts x 16 rows, 6144 x
        // 4096: 127 us; wide tiles 131, pairs 150).
        shape = narrow_ok ? kFpNarrow : kFpWide;
    } else {
        // The shape with the shorter waves.  A tile costs a fixed part and a part per stage, in us, by least squares over
        // 112 products (2 to 32 experts of 160 to 4,096 rows on average, K = 1024 and 6144); an SM takes as long for half a
        // pair's tile as for a wide one, and a launch of pairs starts 0.9 us later.  Experts are taken to spread around
        // their mean as choices at random do.  Of 32 experts, 6144 x 4096: with about 1,024 rows each wide tiles take 707
        // us, pairs 722, narrow ones 797; with about 160 rows 179, 174, 211.  Narrow tiles make the most of few (2 experts
        // x about 1,024 rows, 6144 x 1024: 15.8 us, wide ones 21.9).  On 128 other products (2048 x 2048 to 3584 x 7168)
        // the choice is 0.7 % on average, 13 % at most, behind the best shape.
        const double kb = static_cast<double>(fp_blocks(K));
        const double fixed[3] = {1.46, 1.46, 0.5}, stage[3] = {0.403, 0.403, 0.257}, start[3] = {0.9, 0.0, 0.0};
        const double spread = std::sqrt(avg);
        auto tiles_m = [&](double bm) {
            return (std::ceil((avg - spread) / bm) + std::ceil((avg + spread) / bm)) / 2;
        };
        double best = 1e300;
        shape = kFpWide;
        for (int s2 = kFpPair; s2 <= kFpNarrow; ++s2) {
            if ((s2 == kFpPair && (cap < 2 || want_bm == 128)) || (s2 == kFpNarrow && !narrow_ok)) continue;
            const int units = s2 == kFpPair ? cap / 2 : cap;
            const double tiles = E * tiles_m(s2 == kFpPair ? 256 : 128) * tiles_n(s2);
            const double cost = start[s2] + std::max(1.0, std::ceil(tiles / units)) * (fixed[s2] + stage[s2] * kb);
            if (cost < best) {
                best = cost;
                shape = s2;
            }
        }
    }
    const bool pair = shape == kFpPair;
    const int bm = pair ? 256 : 128;
    if (pair && cap < 2) return RGG_ERR_INVALID_ARG;
    const int64_t most = (M_tot / bm + E) * tiles_n(shape);
    if (most >= (int64_t(1) << 30)) return RGG_ERR_UNSUPPORTED;
    const uint32_t w_bytes = fp_w_bytes(shape);
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
    a.n_tiles_n = tiles_n(shape);
    a.stages = stages;
    a.y_vec32 = (N % 16 == 0 && host_aligned(Y, 32)) ? 1 : 0;
    a.n_major = avg >= 3 * bm ? 1 : 0;  // as the bf16 plan: the tiles that read one weight panel side by side
    a.debug_flags = opt ? (opt->debug_flags & RGG_DEBUG_PRODUCER_STALL) : 0;
    a.timeout_ns = (opt && opt->timeout_ns) ? opt->timeout_ns : kHostDefaultTimeoutNs;
    const int grid = static_cast<int>(pair ? 2 * std::max<int64_t>(1, std::min<int64_t>(cap / 2, most))
                                           : std::max<int64_t>(1, std::min<int64_t>(cap, most)));
    const FpKernel kernels[kFpKernels] = {grouped_fp8_block_pair_kernel<false>, grouped_fp8_block_pair_kernel<true>,
                                          grouped_fp8_block_kernel<kFpWide, false>, grouped_fp8_block_kernel<kFpWide, true>,
                                          grouped_fp8_block_kernel<kFpNarrow, false>};
    const int which = 2 * shape + (gate_up ? 1 : 0);
    cudaError_t err = prepare_fp8_block(kernels[which], which, fp_regs_launch(shape), dev);
    if (err == cudaSuccess) err = launch_chained(kernels[which], grid, fp_threads(shape), smem, st, m, a);
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
