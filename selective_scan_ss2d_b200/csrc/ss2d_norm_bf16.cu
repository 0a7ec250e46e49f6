// ss2d_norm_bf16.cu -- the block norms' kernels for __nv_bfloat16 inputs.
#include "ss2d_norm_launch.cuh"

namespace ss2d {
cudaError_t launch_norm_bf16(const NormParams &p, const NormPlan &pl, bool bwd, bool rf, int grid, int threads,
                            cudaStream_t st)
{
    return rf ? launch_norm_type<__nv_bfloat16, float>(p, pl, bwd, grid, threads, st)
              : launch_norm_type<__nv_bfloat16, __nv_bfloat16>(p, pl, bwd, grid, threads, st);
}
}  // namespace ss2d
