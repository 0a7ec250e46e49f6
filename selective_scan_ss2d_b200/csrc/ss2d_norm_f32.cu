// ss2d_norm_f32.cu -- the block norms' kernels for float inputs, and the sum of the column partials.
#include "ss2d_norm_launch.cuh"

namespace ss2d {
cudaError_t launch_norm_f32(const NormParams &p, const NormPlan &pl, bool bwd, int grid, int threads, cudaStream_t st)
{
    return launch_norm_type<float, float>(p, pl, bwd, grid, threads, st);
}
cudaError_t launch_norm_colsum(const float *part, const NormSums &o, int nparts, int D, cudaStream_t st)
{
    norm_colsum_kernel<<<dim3((D + 31) / 32, kNormCols), 1024, 0, st>>>(part, o, nparts, D);
    return cudaGetLastError();
}
}  // namespace ss2d
