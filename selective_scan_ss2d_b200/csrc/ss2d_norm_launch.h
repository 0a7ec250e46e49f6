// ss2d_norm_launch.h -- internal interface between the block norms' C ABI
// (ss2d_norm.cu) and their kernels, one translation unit per input type.
#pragma once

#include <cuda_runtime.h>

#include "ss2d_norm.cuh"

namespace ss2d {

// values per vector and thread, and the parts that the kernel is compiled for
struct NormPlan {
    int V, E, M;
};
// rf: the residual is float32
cudaError_t launch_norm_f32(const NormParams &p, const NormPlan &pl, bool bwd, int grid, int threads, cudaStream_t st);
cudaError_t launch_norm_bf16(const NormParams &p, const NormPlan &pl, bool bwd, bool rf, int grid, int threads,
                             cudaStream_t st);
cudaError_t launch_norm_f16(const NormParams &p, const NormPlan &pl, bool bwd, bool rf, int grid, int threads,
                            cudaStream_t st);
cudaError_t launch_norm_colsum(const float *part, const NormSums &o, int nparts, int D, cudaStream_t st);

}  // namespace ss2d
