// ss2d_delta_bwd_f16.cu -- the gated delta rule's backward kernels for __half inputs.
#include "ss2d_delta_launch.cuh"

namespace ss2d {
cudaError_t launch_delta_bwd_f16(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    return launch_delta_bwd<__half>(p, pl, st);
}
}  // namespace ss2d
