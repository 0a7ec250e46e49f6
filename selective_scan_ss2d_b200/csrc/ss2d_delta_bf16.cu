// ss2d_delta_bf16.cu -- the gated delta rule's forward kernels for __nv_bfloat16 inputs.
#include "ss2d_delta_launch.cuh"

namespace ss2d {
cudaError_t launch_delta_bf16(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st)
{
    return launch_delta<__nv_bfloat16>(p, pl, what, st);
}
}  // namespace ss2d
