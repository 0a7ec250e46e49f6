// ss2d_norm_f16.cu -- the block norms' kernels for __half inputs.
#include "ss2d_norm_launch.cuh"

namespace ss2d {
cudaError_t launch_norm_f16(const NormParams &p, const NormPlan &pl, bool bwd, bool rf, int grid, int threads,
                            cudaStream_t st)
{
    return rf ? launch_norm_type<__half, float>(p, pl, bwd, grid, threads, st)
              : launch_norm_type<__half, __half>(p, pl, bwd, grid, threads, st);
}
}  // namespace ss2d
