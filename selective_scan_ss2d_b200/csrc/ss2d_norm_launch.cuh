// ss2d_norm_launch.cuh -- launches of the block norms for one input type.
#pragma once

#include "ss2d_norm_launch.h"

namespace ss2d {

template <typename Tin, typename Tr, int V, int E, int M>
cudaError_t launch_norm_parts(const NormParams &p, bool bwd, int grid, int threads, cudaStream_t st)
{
    if (!bwd) {
        norm_fwd_kernel<Tin, Tr, V, E, M><<<grid, threads, 0, st>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {(unsigned)grid, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = sizeof(float) * threads * E;
    cfg.stream = st;
    if (p.cols && !p.part) {   // one cluster, which sums its CTAs' columns
        cfg.dynamicSmemBytes += sizeof(float) * kNormCols * p.D;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
    }
    if constexpr (M == kNormAny || (M & kHasBias)) {
        if (p.cols >> 3)
            return cudaLaunchKernelEx(&cfg, norm_bwd_kernel<Tin, Tr, V, E, true, M>, p);
    }
    return cudaLaunchKernelEx(&cfg, norm_bwd_kernel<Tin, Tr, V, E, false, M>, p);
}
template <typename Tin, typename Tr, int V, int E>
cudaError_t launch_norm_full(const NormParams &p, int M, bool bwd, int grid, int threads, cudaStream_t st)
{
    switch (M) {
    case kHasPost:
        return launch_norm_parts<Tin, Tr, V, E, kHasPost>(p, bwd, grid, threads, st);
    case kHasPost | kHasGate:
        return launch_norm_parts<Tin, Tr, V, E, kHasPost | kHasGate>(p, bwd, grid, threads, st);
    case kHasRes | kHasPre:
        return launch_norm_parts<Tin, Tr, V, E, kHasRes | kHasPre>(p, bwd, grid, threads, st);
    case kHasRes | kHasPre | kHasScale | kHasBias:
        return launch_norm_parts<Tin, Tr, V, E, kHasRes | kHasPre | kHasScale | kHasBias>(p, bwd, grid, threads, st);
    default:
        return launch_norm_parts<Tin, Tr, V, E, kHasPost | kHasGate | kHasRes | kHasPre | kHasScale>(p, bwd, grid,
                                                                                                    threads, st);
    }
}
template <typename Tin, typename Tr>
cudaError_t launch_norm_type(const NormParams &p, const NormPlan &pl, bool bwd, int grid, int threads,
                             cudaStream_t st)
{
    if (pl.M != kNormAny)
        return pl.E == 12 ? launch_norm_full<Tin, Tr, 4, 12>(p, pl.M, bwd, grid, threads, st)
                          : launch_norm_full<Tin, Tr, 8, 8>(p, pl.M, bwd, grid, threads, st);
    if (pl.E == 16)
        return pl.V == 8 ? launch_norm_parts<Tin, Tr, 8, 16, kNormAny>(p, bwd, grid, threads, st)
                         : launch_norm_parts<Tin, Tr, 1, 16, kNormAny>(p, bwd, grid, threads, st);
    return pl.V == 8 ? launch_norm_parts<Tin, Tr, 8, 8, kNormAny>(p, bwd, grid, threads, st)
                     : launch_norm_parts<Tin, Tr, 1, 8, kNormAny>(p, bwd, grid, threads, st);
}

}  // namespace ss2d
