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

// chains of a pass: segments (every slot that may hold one), or sequences
inline long long delta_units(const DeltaParams &p)
{
    if (!p.SC)
        return p.nseq;
    return p.cu ? p.nslots / p.SC + p.nseq : (long long)p.nseq * ((p.NC + p.SC - 1) / p.SC);
}

template <typename Tin, int DKP, int NW, int NP, int NPP, int STAGES>
cudaError_t launch_out(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, NW, kChainOut, NP, NPP, STAGES>::bytes;
    auto kern = delta_out_kernel<Tin, DKP, NW, NP, NPP, STAGES>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    const long long units = delta_units(p);
    const dim3 grid((p.DV + NW * 16 - 1) / (NW * 16), p.H, (unsigned)(units < 65535 ? units : 65535));
    kern<<<grid, NW * 32, smem, st>>>(p, units);
    return cudaGetLastError();
}
template <typename Tin, int DKP, int NW, int STAGES>
cudaError_t launch_both(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, NW, kChainRev, 3, 3, STAGES>::bytes;
    auto kern = delta_both_kernel<Tin, DKP, NW, STAGES>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    const long long units = delta_units(p);
    const dim3 grid(2 * ((p.DV + NW * 16 - 1) / (NW * 16)), p.H, (unsigned)(units < 65535 ? units : 65535));
    kern<<<grid, NW * 32, smem, st>>>(p, units);
    return cudaGetLastError();
}

// Stages that fit: a second one hides the next chunk's copies behind this chunk's
// products; one leaves room for a second and third CTA, which hide them too.
constexpr int chain_stages(int two_bytes) { return two_bytes <= 225 * 1024 ? 2 : 1; }

// CTAs of four warps (64 columns of DV).  With more of them than two per SM, a
// single stage and up to three CTAs per SM; otherwise two stages if they fit.
template <typename Tin, int DKP, int NP, int NPP>
cudaError_t launch_chain_out(const DeltaParams &p, cudaStream_t st)
{
    const long long ctas = (long long)((p.DV + 63) / 64) * p.H * delta_units(p);
    constexpr int two = chain_stages(ChainLayout<Tin, DKP, 4, kChainOut, NP, NPP, 2>::bytes);
    if (two == 1 || ctas > 2 * 148)
        return launch_out<Tin, DKP, 4, NP, NPP, 1>(p, st);
    return launch_out<Tin, DKP, 4, NP, NPP, two>(p, st);
}
template <typename Tin, int DKP, int MODE>
cudaError_t launch_one(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, 4, MODE, 3, 3, 1>::bytes;
    auto kern = delta_one_kernel<Tin, DKP, 4, 1, MODE>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    const long long units = delta_units(p);
    kern<<<dim3((p.DV + 63) / 64, p.H, (unsigned)(units < 65535 ? units : 65535)), 128, smem, st>>>(p, units);
    return cudaGetLastError();
}
// Both chains of a backward pass in one launch while they do not fill the SMs
// twice; beyond that one after the other: CTAs of both on an SM wait for
// instructions (6144 chunks of 64 x 64 heads: 3 of 10 cycles a warp waited).
template <typename Tin, int DKP>
cudaError_t launch_chain_both(const DeltaParams &p, cudaStream_t st)
{
    const long long ctas = (long long)((p.DV + 63) / 64) * p.H * delta_units(p) * 2;
    if (ctas > 2 * 148) {
        const cudaError_t e = launch_one<Tin, DKP, kChainState>(p, st);
        return e != cudaSuccess ? e : launch_one<Tin, DKP, kChainRev>(p, st);
    }
    constexpr int two = chain_stages(ChainLayout<Tin, DKP, 4, kChainRev, 3, 3, 2>::bytes);
    return launch_both<Tin, DKP, 4, two>(p, st);
}

// the segments' ends and the states that they start from (REV: and end with in reverse)
template <typename Tin, int DKP, int NP, bool REV>
cudaError_t launch_segments(const DeltaParams &p, cudaStream_t st)
{
    constexpr int MODE = REV ? kChainRev : kChainState;   // the larger layout of the pass
    constexpr int stages = chain_stages(2 * ChainLayout<Tin, DKP, 4, MODE, NP, 3, 2>::bytes);
    constexpr int smem = ChainLayout<Tin, DKP, 4, MODE, NP, 3, stages>::bytes;
    auto kern = delta_local_kernel<Tin, DKP, NP, stages, REV>;
    cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    const int dvt = (p.DV + 63) / 64, dkt = (p.DK + 63) / 64;
    const long long units = delta_units(p);
    kern<<<dim3(dvt * (REV ? 2 : 1) + dkt, p.H, (unsigned)(units < 65535 ? units : 65535)), 128, smem, st>>>(p, dvt, dkt,
                                                                                                          units);
    e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    using CL = CombineLayout<DKP>;
    auto comb = delta_combine_kernel<DKP, REV>;
    e = delta_smem(comb, CL::bytes);
    if (e != cudaSuccess)
        return e;
    comb<<<dim3(p.DV / 16 * (REV ? 2 : 1), p.H, p.nseq < 65535 ? p.nseq : 65535), CL::threads, CL::bytes, st>>>(p);
    return cudaGetLastError();
}

template <typename Tin, int DKP, bool SHARED>
cudaError_t launch_grad(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = GradLayout<Tin, DKP>::bytes;
    auto kern = delta_grad_kernel<Tin, DKP, SHARED>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<dim3((unsigned)p.nslots, p.HK), kGradThreads, smem, st>>>(p);
    return cudaGetLastError();
}

template <typename Tin, int DKP>
cudaError_t launch_bwd(const DeltaParams &p, cudaStream_t st)
{
    cudaError_t e = launch_prep<Tin, DKP, 3, 3>(p, st);
    if (e == cudaSuccess && p.SC)
        e = launch_segments<Tin, DKP, 3, true>(p, st);
    if (e == cudaSuccess)
        e = launch_chain_both<Tin, DKP>(p, st);
    if (e != cudaSuccess)
        return e;
    return p.H > p.HK ? launch_grad<Tin, DKP, true>(p, st) : launch_grad<Tin, DKP, false>(p, st);
}

template <typename Tin, int DKP, int NP, int NPP>
cudaError_t launch_fwd_parts(const DeltaParams &p, cudaStream_t st)
{
    cudaError_t e = launch_prep<Tin, DKP, NP, NPP>(p, st);
    if (e == cudaSuccess && p.SC)
        e = launch_segments<Tin, DKP, NP, false>(p, st);
    return e != cudaSuccess ? e : launch_chain_out<Tin, DKP, NP, NPP>(p, st);
}
template <typename Tin, int DKP>
cudaError_t launch_fwd(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    if constexpr (sizeof(Tin) == 4)
        return launch_fwd_parts<Tin, DKP, 3, 3>(p, st);
    else
        return pl.np == 3 ? launch_fwd_parts<Tin, DKP, 3, 2>(p, st) : launch_fwd_parts<Tin, DKP, 2, 2>(p, st);
}

// Columns of a state per CTA: 64 (or all), fewer while that leaves SMs without
// work.  CTAs of 128 columns (16 rows of four to a thread, two CTAs per SM) took
// 123 us for 4096 states of 128 x 128.
template <typename Tin>
cudaError_t launch_recur(const DeltaParams &p, cudaStream_t st)
{
    int dvt = p.DV < 64 ? p.DV : 64;
    while (dvt > 16 && dvt % 32 == 0 && (long long)((p.DV + dvt - 1) / dvt) * p.H * p.nseq < 148)
        dvt /= 2;
    const dim3 grid((p.DV + dvt - 1) / dvt, p.H, p.nseq < 65535 ? p.nseq : 65535);
    // rows per thread: DK over the row groups of 256 threads
    const int rows = (p.DK + kRecurThreads / (dvt / 4) - 1) / (kRecurThreads / (dvt / 4));
    if (rows <= 4)
        delta_recur_kernel<Tin, 4><<<grid, kRecurThreads, 0, st>>>(p, dvt);
    else
        delta_recur_kernel<Tin, 8><<<grid, kRecurThreads, 0, st>>>(p, dvt);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_delta(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st)
{
    if (what == kDeltaRecur)
        return launch_recur<Tin>(p, st);
    return pl.dkp == 64 ? launch_fwd<Tin, 64>(p, pl, st) : launch_fwd<Tin, 128>(p, pl, st);
}
template <typename Tin>
cudaError_t launch_delta_bwd(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st)
{
    return pl.dkp == 64 ? launch_bwd<Tin, 64>(p, st) : launch_bwd<Tin, 128>(p, st);
}

}  // namespace ss2d
