// ss2d_delta_bwd_bf16.cu -- the gated delta rule's backward kernels for __nv_bfloat16 inputs.
#include "ss2d_delta_launch.cuh"

namespace ss2d {
cudaError_t launch_delta_bwd_bf16(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    return launch_delta_bwd<__nv_bfloat16>(p, pl, st);
}
}  // namespace ss2d
