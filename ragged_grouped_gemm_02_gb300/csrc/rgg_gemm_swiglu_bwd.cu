// The backward pass of the fused gate-up projection with SiLU (epilogue
// kEpiSwiGLUBwd): gate and up are computed again on the forward op's tiles and
// the epilogue turns them and dH into [dGate | dUp] and H, so neither the gate
// nor the up product is ever stored.  Bound by the MMAs at many rows (32,768 rows,
// K = 6144, N = 2048: 945 us, 1 746 TFLOP/s), by bytes at few: 64 experts x 256
// rows, K = 1024, N = 1344 takes 99 us at 5.7 TB/s (134 us while dH was read
// after the accumulators were ready and outputs went out 16 bytes at a time).
// Few tiles are 64 x 128, as for the gradient by the activations.
#include "rgg_gemm_launch.cuh"

namespace rgg {

cudaError_t launch_gemm_swiglu_bwd(int bm, int bn, int grid, size_t smem, cudaStream_t stream,
                                   const CUtensorMap& tmap_x, const CUtensorMap& tmap_x64, const CUtensorMap& tmap_w,
                                   const GemmArgs& args) {
    if (bm == 64 && bn == 128)
        return launch_gemm_instance<64, 128, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 64 && bn == 256)
        return launch_gemm_instance<64, 256, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 128 && bn == 128)
        return launch_gemm_instance<128, 128, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 128 && bn == 256)
        return launch_gemm_instance<128, 256, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 256 && bn == 128)
        return launch_pair_instance<128, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    if (bm == 256 && bn == 256)
        return launch_pair_instance<256, kEpiSwiGLUBwd>(grid, smem, stream, tmap_x, tmap_x64, tmap_w, args);
    return cudaErrorInvalidValue;
}

cudaError_t launch_gemm_mixed_swiglu_bwd(int pair_grid, size_t pair_smem, const GemmArgs& pair_args, int single_grid,
                                         size_t single_smem, const GemmArgs& single_args, cudaStream_t stream,
                                         const CUtensorMap& tmap_x, const CUtensorMap& tmap_x64,
                                         const CUtensorMap& tmap_w) {
    return launch_mixed_instance<kEpiSwiGLUBwd>(pair_grid, pair_smem, pair_args, single_grid, single_smem, single_args,
                                                stream, tmap_x, tmap_x64, tmap_w);
}

}  // namespace rgg
