// rgg_moe.cu -- a serving step of a mixture-of-experts layer with 8-bit experts in one call: the operators' own entry
// points one behind the other, their results between them in a caller's workspace.
//
// For a few tokens the step is a chain of short launches; queued from one call they follow each other without gaps (16
// tokens, 64 experts of 1024 x 1408: 88 us through six calls from Python, of which the GPU is busy for 55).
#include <algorithm>

#include "rgg_fp8_block.h"
#include "rgg_host.h"
#include "rgg_internal.h"

namespace rgg {

// Where each result lies in the workspace, from its start.
struct MoePlan {
    int64_t experts, weights, offsets, row_index, position, sort, sort_bytes, x_codes, x_scales, h_codes, h_scales, y, total;
};

static MoePlan moe_plan(int64_t T, int E, int k, int K, int N, int K_out) {
    MoePlan p;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t rows = T * k;
    p.experts = take(4 * rows);
    p.weights = take(4 * rows);
    p.offsets = take(4 * (static_cast<int64_t>(E) + 1));
    p.row_index = take(4 * rows);
    p.position = take(4 * rows);
    p.sort_bytes = rgg_sort_by_expert_workspace(rows, E);
    p.sort = take(p.sort_bytes);
    p.x_codes = take(rows * K);
    p.x_scales = take(4 * rows * fp_blocks(K));
    p.h_codes = take(rows * N);
    p.h_scales = take(4 * rows * fp_blocks(N));
    p.y = take(2 * rows * K_out);
    p.total = at;
    return p;
}

static bool moe_sizes_ok(int64_t T, int E, int k, int K, int N, int K_out) {
    const int64_t most = int64_t(1) << 31;
    if (T < 0 || T >= most || k < 1 || T * k >= most || T * k * std::max(K, std::max(N, K_out)) >= int64_t(1) << 56)
        return false;  // the last: the workspace's size is counted in 64 bits
    return k <= E && K % 16 == 0 && N % kFpBlock == 0 &&
           N <= kMaxWidth / 2 && host_check_sizes(E, T * k, K, N) == RGG_OK && host_check_sizes(E, T * k, N, K_out) == RGG_OK;
}

}  // namespace rgg

using namespace rgg;

extern "C" int64_t rgg_moe_swiglu_fp8_block_workspace(int64_t T, int E, int k, int K, int N, int K_out) {
    return moe_sizes_ok(T, E, k, K, N, K_out) ? moe_plan(T, E, k, K, N, K_out).total : 0;
}

extern "C" rgg_status rgg_moe_swiglu_fp8_block(rgg_handle* h, const void* X, const void* logits, int logits_dtype,
                                               const void* w13_codes, const float* w13_scales, const void* w2_codes,
                                               const float* w2_scales, void* out, int64_t T, int E, int k, int K, int N,
                                               int K_out, int flags, float scale, void* workspace,
                                               int64_t workspace_bytes, void* stream) {
    if (!h || !w13_codes || !w13_scales || !w2_codes || !w2_scales) return RGG_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > 32) return RGG_ERR_UNSUPPORTED;
    if (!moe_sizes_ok(T, E, k, K, N, K_out)) return RGG_ERR_INVALID_ARG;
    if (flags & ~(RGG_ROUTE_SIGMOID | RGG_ROUTE_RENORMALIZE) || scale != scale) return RGG_ERR_INVALID_ARG;
    if (logits_dtype != RGG_BF16 && logits_dtype != RGG_FP32 && logits_dtype != RGG_FP16) return RGG_ERR_INVALID_ARG;
    if (!host_aligned(w13_codes, 16) || !host_aligned(w13_scales, 4) || !host_aligned(w2_codes, 16) ||
        !host_aligned(w2_scales, 4))
        return RGG_ERR_INVALID_ARG;
    if (T == 0) return RGG_OK;
    if (!X || !logits || !out || !workspace || !host_aligned(X, 16) || !host_aligned(out, 2) ||
        !host_aligned(workspace, 256) || !host_aligned(logits, logits_dtype == RGG_FP32 ? 4 : 2))
        return RGG_ERR_INVALID_ARG;
    const MoePlan p = moe_plan(T, E, k, K, N, K_out);
    if (workspace_bytes < p.total) return RGG_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto ints = [&](int64_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    auto floats = [&](int64_t at) { return reinterpret_cast<float*>(ws + at); };
    const int64_t rows = T * k;
    rgg_status s = rgg_route_topk(h, logits, logits_dtype, T, E, k, flags, scale, ints(p.experts), floats(p.weights), stream);
    if (s == RGG_OK)
        s = rgg_sort_by_expert(h, ints(p.experts), T, k, E, ints(p.offsets), ints(p.row_index), ints(p.position),
                               ws + p.sort, p.sort_bytes, stream);
    if (s == RGG_OK)
        s = rgg_fp8_block_quantize(h, X, ints(p.position), T, k, rows, K, ws + p.x_codes, floats(p.x_scales), stream);
    if (s == RGG_OK)
        s = rgg_grouped_gemm_swiglu_fp8_block(h, ws + p.x_codes, floats(p.x_scales), w13_codes, w13_scales,
                                              ints(p.offsets), ws + p.h_codes, floats(p.h_scales), E, rows, K, N, stream,
                                              nullptr);
    if (s == RGG_OK)
        s = rgg_grouped_gemm_fp8_block(h, ws + p.h_codes, floats(p.h_scales), w2_codes, w2_scales, ints(p.offsets),
                                       ws + p.y, E, rows, N, K_out, stream, nullptr);
    if (s == RGG_OK)
        s = rgg_combine(h, ws + p.y, ints(p.position), floats(p.weights), T, k, rows, K_out, out, stream);
    return s;
}
