// ss2d_delta_f32.cu -- the gated delta rule's forward kernels for float inputs.
#include "ss2d_delta_launch.cuh"

namespace ss2d {
cudaError_t launch_delta_f32(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st)
{
    return launch_delta<float>(p, pl, what, st);
}
}  // namespace ss2d
