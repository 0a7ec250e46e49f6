// ss2d_delta_launch.cuh -- kernel choice and launches of the gated delta rule
// for one input type.
#pragma once

#include "ss2d_delta_chain.cuh"
#include "ss2d_delta_grad.cuh"
#include "ss2d_delta_launch.h"

namespace ss2d {

template <typename... A>
cudaError_t delta_smem(void (*kern)(A...), int bytes)
{
    return bytes > 32 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                             : cudaSuccess;
}

template <typename Tin, int DKP, int NPT, int NPP>
cudaError_t launch_prep(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = PrepLayout<DKP, DeltaParts<Tin>::n, NPT, NPP>::bytes;
    auto kern = delta_prep_kernel<Tin, DKP, NPT, NPP>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<dim3((unsigned)p.nslots, p.HK), kPrepThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename Tin, int DKP, int NW, int MODE, int NP, int NPP>
cudaError_t launch_chain_nw(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, NW, MODE, NP, NPP>::bytes;
    auto kern = delta_chain_kernel<Tin, DKP, NW, MODE, NP, NPP>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((p.DV + NW * 16 - 1) / (NW * 16), p.H, p.nseq < 65535 ? p.nseq : 65535);
    kern<<<grid, NW * 32, smem, st>>>(p);
    return cudaGetLastError();
}

// Eight warps (128 columns of DV) share a chunk's K, Q, T and P when there
// are enough such CTAs for every SM; otherwise four warps, one per scheduler,
// on twice as many SMs.
template <typename Tin, int DKP, int MODE, int NP, int NPP>
cudaError_t launch_chain(const DeltaParams &p, cudaStream_t st)
{
    const long long wide = (long long)((p.DV + 127) / 128) * p.H * p.nseq;
    if (p.DV > 64 && wide >= 148)
        return launch_chain_nw<Tin, DKP, 8, MODE, NP, NPP>(p, st);
    return launch_chain_nw<Tin, DKP, 4, MODE, NP, NPP>(p, st);
}

template <typename Tin, int DKP>
cudaError_t launch_bwd(const DeltaParams &p, cudaStream_t st)
{
    cudaError_t e = launch_prep<Tin, DKP, 3, 3>(p, st);
    if (e == cudaSuccess)
        e = launch_chain<Tin, DKP, kChainState, 3, 3>(p, st);
    if (e == cudaSuccess)
        e = launch_chain<Tin, DKP, kChainRev, 3, 3>(p, st);
    if (e != cudaSuccess)
        return e;
    constexpr int smem = GradLayout<Tin, DKP>::bytes;
    auto kern = delta_grad_kernel<Tin, DKP>;
    e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<dim3((unsigned)p.nslots, p.HK), kGradThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename Tin, int DKP>
cudaError_t launch_fwd(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    cudaError_t e;
    if constexpr (sizeof(Tin) == 4) {
        e = launch_prep<Tin, DKP, 3, 3>(p, st);
        return e != cudaSuccess ? e : launch_chain<Tin, DKP, kChainOut, 3, 3>(p, st);
    } else {
        if (pl.np == 3) {
            e = launch_prep<Tin, DKP, 3, 2>(p, st);
            return e != cudaSuccess ? e : launch_chain<Tin, DKP, kChainOut, 3, 2>(p, st);
        }
        e = launch_prep<Tin, DKP, 2, 2>(p, st);
        return e != cudaSuccess ? e : launch_chain<Tin, DKP, kChainOut, 2, 2>(p, st);
    }
}

// Columns of a state per CTA: 128 (or all), fewer while that leaves SMs without work.
template <typename Tin>
cudaError_t launch_recur(const DeltaParams &p, cudaStream_t st)
{
    int dvt = p.DV < 128 ? p.DV : 128;
    while (dvt > 16 && dvt % 32 == 0 && (long long)((p.DV + dvt - 1) / dvt) * p.H * p.nseq < 148)
        dvt /= 2;
    const dim3 grid((p.DV + dvt - 1) / dvt, p.H, p.nseq < 65535 ? p.nseq : 65535);
    delta_recur_kernel<Tin><<<grid, kRecurThreads, 0, st>>>(p, dvt);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_delta(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st)
{
    if (what == kDeltaRecur)
        return launch_recur<Tin>(p, st);
    if (what == kDeltaFwd)
        return pl.dkp == 64 ? launch_fwd<Tin, 64>(p, pl, st) : launch_fwd<Tin, 128>(p, pl, st);
    return pl.dkp == 64 ? launch_bwd<Tin, 64>(p, st) : launch_bwd<Tin, 128>(p, st);
}

}  // namespace ss2d
