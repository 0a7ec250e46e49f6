// ss2d_delta_bwd_f32.cu -- the gated delta rule's backward kernels for float inputs.
#include "ss2d_delta_launch.cuh"

namespace ss2d {
cudaError_t launch_delta_bwd_f32(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    return launch_delta_bwd<float>(p, pl, st);
}
}  // namespace ss2d
