// The mixed launch (rgg_sched.cuh): 256-row tiles of the large experts on CTA
// pairs beside 128-row tiles of the small ones on single CTAs, two kernels on
// disjoint SMs that claim tiles from the same two device counters.
#include "rgg_gemm_launch.cuh"

namespace rgg {

cudaError_t launch_gemm_mixed(int pair_grid, size_t pair_smem, const GemmArgs& pair_args, int single_grid,
                              size_t single_smem, const GemmArgs& single_args, cudaStream_t stream,
                              const CUtensorMap& tmap_x, const CUtensorMap& tmap_x64, const CUtensorMap& tmap_w) {
    return launch_mixed_instance<kEpiPlain>(pair_grid, pair_smem, pair_args, single_grid, single_smem, single_args,
                                            stream, tmap_x, tmap_x64, tmap_w);
}

cudaError_t launch_gemm_mixed_swiglu(int pair_grid, size_t pair_smem, const GemmArgs& pair_args, int single_grid,
                                     size_t single_smem, const GemmArgs& single_args, cudaStream_t stream,
                                     const CUtensorMap& tmap_x, const CUtensorMap& tmap_x64,
                                     const CUtensorMap& tmap_w) {
    return launch_mixed_instance<kEpiSwiGLU>(pair_grid, pair_smem, pair_args, single_grid, single_smem, single_args,
                                             stream, tmap_x, tmap_x64, tmap_w);
}

}  // namespace rgg
