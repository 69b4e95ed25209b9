// The gradient by the activations, dX_e = dY_e . W_e^T: the grouped product with
// W read as it lies (kTransW, a K-major B operand), on every tile shape of the
// forward product.  What bounds it is what bounds the forward product: the
// same bytes per stage, MMAs and epilogue.  32 experts, 32,768 rows, K = 6144,
// N = 4096: 922 us from a pause (1 788 TFLOP/s), 1 092 us in a row at the power
// cap; the forward product of the same size 916.  Few reduction stages are bound
// by the stores (epilogue_groups), few tiles by the weights each SM streams,
// which the narrowest tiles make least (few_tiles_options).
#include "rgg_gemm_launch.cuh"

namespace rgg {

template <int BM>
static cudaError_t launch_dgrad_single(int bn, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& tmap_x,
                                       const CUtensorMap& tmap_x64, const CUtensorMap& tmap_w, const GemmArgs& args) {
    switch (bn) {
        case 128:
            return launch_gemm_instance<BM, 128, kEpiPlain, false, kGatherNone, true>(grid, smem, stream, tmap_x,
                                                                                      tmap_x64, tmap_w, args);
        case 192:
            return launch_gemm_instance<BM, 192, kEpiPlain, false, kGatherNone, true>(grid, smem, stream, tmap_x,
                                                                                      tmap_x64, tmap_w, args);
        case 256:
            return launch_gemm_instance<BM, 256, kEpiPlain, false, kGatherNone, true>(grid, smem, stream, tmap_x,
                                                                                      tmap_x64, tmap_w, args);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gemm_dgrad(int bm, int bn, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& tmap_x,
                              const CUtensorMap& tmap_x64, const CUtensorMap& tmap_w, const GemmArgs& args) {
    if (bm == 64) return launch_dgrad_single<64>(bn, grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 128) return launch_dgrad_single<128>(bn, grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 256 && bn == 128)
        return launch_pair_instance<128, kEpiPlain, true>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 256 && bn == 256)
        return launch_pair_instance<256, kEpiPlain, true>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    return cudaErrorInvalidValue;
}

cudaError_t launch_gemm_mixed_dgrad(int pair_grid, size_t pair_smem, const GemmArgs& pair_args, int single_grid,
                                    size_t single_smem, const GemmArgs& single_args, cudaStream_t stream,
                                    const CUtensorMap& tmap_x, const CUtensorMap& tmap_x64,
                                    const CUtensorMap& tmap_w) {
    return launch_mixed_instance<kEpiPlain, true>(pair_grid, pair_smem, pair_args, single_grid, single_smem,
                                                  single_args, stream, tmap_x, tmap_x64, tmap_w);
}

}  // namespace rgg
