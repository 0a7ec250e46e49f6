// ss2d_delta_launch.cuh -- kernel choice and launches of the gated delta rule
// for one input type.
#pragma once

#include "ss2d_delta_chain.cuh"
#include "ss2d_delta_grad.cuh"
#include "ss2d_delta_launch.h"
#include "ss2d_delta_split.cuh"

namespace ss2d {

template <typename... A>
cudaError_t delta_smem(void (*kern)(A...), int bytes)
{
    return bytes > 32 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)
                             : cudaSuccess;
}

// Which form a chain takes.  Many chains (more than kWideCtas CTAs): one warp to 16
// columns, one stage, two or three CTAs per SM.  Few: one warp with two stages for
// heads of up to 64 in 16 bits (4.4 us a chunk against 5.1 with four warps), four warps for
// wider heads and float32 (both chains of 4096 tokens, 128 x 128: 533 us against 621; seven
// float32 sequences of 32 x 64: 67 against 100).  float16, whose one-warp form has fewer products,
// takes four warps, and k and q in parts, only for the outputs of few wide heads (a call on 4096 tokens, 32
// chains: 388 us against 488; 500 tokens, 128 chains 151 against 107; a backward pass of 32 chains 1298 against
// 1087, 16384 tokens of 4 heads in segments 291 against 217).
template <typename Tin, int DKP>
constexpr bool chain_split_out() { return sizeof(Tin) == 4 || DKP == 128; }
template <typename Tin, int DKP>
constexpr bool chain_split() { return sizeof(Tin) == 4 || (DKP == 128 && !std::is_same_v<Tin, __half>); }

template <typename Tin, int DKP, int NPT, int NPP, bool PARTS>
cudaError_t launch_prep_as(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = PrepLayout<DKP, PARTS ? DeltaParts<Tin>::n : 1, NPT, NPP>::bytes;
    auto kern = delta_prep_kernel<Tin, DKP, NPT, NPP, PARTS>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<dim3((unsigned)p.nslots, p.HK), kPrepThreads, smem, st>>>(p);
    return cudaGetLastError();
}

inline dim3 chain_grid(const DeltaParams &p, int tiles)
{
    const long long units = delta_units(p);
    return dim3(tiles, p.H, (unsigned)(units < 65535 ? units : 65535));
}

// p.kp: the chain reads k and q in bf16 parts
template <typename Tin, int DKP, int NPT, int NPP>
cudaError_t launch_prep(const DeltaParams &p, cudaStream_t st)
{
    if constexpr (sizeof(Tin) == 4)
        return launch_prep_as<Tin, DKP, NPT, NPP, true>(p, st);
    else if constexpr (chain_split_out<Tin, DKP>() && std::is_same_v<Tin, __half> && NPP == 2)
        return p.kp ? launch_prep_as<Tin, DKP, NPT, NPP, true>(p, st) : launch_prep_as<Tin, DKP, NPT, NPP, false>(p, st);
    else
        return launch_prep_as<Tin, DKP, NPT, NPP, false>(p, st);
}

// ---- one warp to 16 columns of DV, CTAs of 64 columns
template <typename Tin, int DKP, int NP, int NPP, int STAGES>
cudaError_t launch_wide_out(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, 4, kChainOut, NP, NPP, STAGES>::bytes;
    auto kern = delta_out_kernel<Tin, DKP, 4, NP, NPP, STAGES>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<chain_grid(p, (p.DV + 63) / 64), 128, smem, st>>>(p, delta_units(p));
    return cudaGetLastError();
}
template <typename Tin, int DKP>
cudaError_t launch_wide_each(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, 4, kChainRev, 3, 3, 1>::bytes;   // the larger of the two
    auto kern = delta_each_kernel<Tin, DKP, 4, 1>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    dim3 grid = chain_grid(p, (p.DV + 63) / 64);
    grid.z = 2 * (grid.z < 32767 ? grid.z : 32767);
    kern<<<grid, 128, smem, st>>>(p, delta_units(p));
    return cudaGetLastError();
}
template <typename Tin, int DKP>
cudaError_t launch_wide_both(const DeltaParams &p, cudaStream_t st)
{
    constexpr int smem = ChainLayout<Tin, DKP, 4, kChainRev, 3, 3, 2>::bytes;
    auto kern = delta_both_kernel<Tin, DKP, 4, 2>;
    const cudaError_t e = delta_smem(kern, smem);
    if (e != cudaSuccess)
        return e;
    kern<<<chain_grid(p, 2 * ((p.DV + 63) / 64)), 128, smem, st>>>(p, delta_units(p));
    return cudaGetLastError();
}

// ---- four warps to 16 columns: four groups to a CTA and two buffers of K where they fit
template <typename Tin, int DKP, int MODE, int NP, int NPP, int MOST = 4>
struct SplitShape {
    static constexpr int most = 226 * 1024;
    static constexpr int groups = SplitLayout<Tin, DKP, 4, MODE, NP, NPP, 2>::bytes <= most ? MOST : 2;
    static constexpr int kbuf = SplitLayout<Tin, DKP, groups, MODE, NP, NPP, 2>::bytes <= most ? 2 : 1;
    static constexpr int bytes = SplitLayout<Tin, DKP, groups, MODE, NP, NPP, kbuf>::bytes;
    static_assert(bytes <= most, "shared memory");
    static int tiles(int n) { return (n + groups * 16 - 1) / (groups * 16); }
};
template <typename Tin, int DKP, int NP, int NPP, int MOST = 4>
cudaError_t launch_split_out(const DeltaParams &p, cudaStream_t st)
{
    using Sh = SplitShape<Tin, DKP, kChainOut, NP, NPP, MOST>;
    // two groups to a CTA while each has an SM (bfloat16, 4096 tokens, 32 chains of 128 x 128: 467 -> 313 us a call)
    if constexpr (MOST == 4 && Sh::groups == 4) {
        if (2 * (long long)Sh::tiles(p.DV) * p.H * delta_units(p) <= 148)
            return launch_split_out<Tin, DKP, NP, NPP, 2>(p, st);
    }
    auto kern = delta_split_out_kernel<Tin, DKP, Sh::groups, NP, NPP, Sh::kbuf>;
    const cudaError_t e = delta_smem(kern, Sh::bytes);
    if (e != cudaSuccess)
        return e;
    kern<<<chain_grid(p, Sh::tiles(p.DV)), Sh::groups * 128, Sh::bytes, st>>>(p, delta_units(p));
    return cudaGetLastError();
}
template <typename Tin, int DKP, int MOST = 4>
cudaError_t launch_split_both(const DeltaParams &p, cudaStream_t st)
{
    using Sh = SplitShape<Tin, DKP, kChainRev, 3, 3, MOST>;   // the larger of the two
    if constexpr (MOST == 4 && Sh::groups == 4) {
        if (4 * (long long)Sh::tiles(p.DV) * p.H * delta_units(p) <= 148)
            return launch_split_both<Tin, DKP, 2>(p, st);
    }
    auto kern = delta_split_both_kernel<Tin, DKP, Sh::groups, Sh::kbuf>;
    const cudaError_t e = delta_smem(kern, Sh::bytes);
    if (e != cudaSuccess)
        return e;
    kern<<<chain_grid(p, 2 * Sh::tiles(p.DV)), Sh::groups * 128, Sh::bytes, st>>>(p, delta_units(p));
    return cudaGetLastError();
}

// the segments' ends and the states that they start from (REV: and end with in reverse)
template <typename Tin, int DKP, int NP, bool REV>
cudaError_t launch_segments(const DeltaParams &p, cudaStream_t st)
{
    constexpr int MODE = REV ? kChainRev : kChainState;   // the larger layout of the pass
    cudaError_t e;
    if constexpr (chain_split<Tin, DKP>()) {
        using Sh = SplitShape<Tin, DKP, MODE, NP, 3>;
        auto kern = delta_split_local_kernel<Tin, DKP, Sh::groups, NP, Sh::kbuf, REV>;
        e = delta_smem(kern, Sh::bytes);
        if (e != cudaSuccess)
            return e;
        const int dvt = Sh::tiles(p.DV), dkt = Sh::tiles(p.DK);
        kern<<<chain_grid(p, dvt * (REV ? 2 : 1) + dkt), Sh::groups * 128, Sh::bytes, st>>>(p, dvt, dkt,
                                                                                           delta_units(p));
    } else {
        // two stages where two such CTAs fit an SM
        constexpr int two = ChainLayout<Tin, DKP, 4, MODE, NP, 3, 2>::bytes;
        constexpr int stages = 2 * two <= 225 * 1024 ? 2 : 1;
        constexpr int smem = ChainLayout<Tin, DKP, 4, MODE, NP, 3, stages>::bytes;
        auto kern = delta_local_kernel<Tin, DKP, NP, stages, REV>;
        e = delta_smem(kern, smem);
        if (e != cudaSuccess)
            return e;
        const int dvt = (p.DV + 63) / 64, dkt = (p.DK + 63) / 64;
        kern<<<chain_grid(p, dvt * (REV ? 2 : 1) + dkt), 128, smem, st>>>(p, dvt, dkt, delta_units(p));
    }
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

template <typename Tin, int DKP, int NP, int NPP>
cudaError_t launch_chain_out(const DeltaParams &p, cudaStream_t st)
{
    if (delta_wide(p, false))
        return launch_wide_out<Tin, DKP, NP, NPP, 1>(p, st);
    if constexpr (chain_split_out<Tin, DKP>()) {
        if (chain_split<Tin, DKP>() || delta_split_f16(p))
            return launch_split_out<Tin, DKP, NP, NPP>(p, st);
    }
    if constexpr (!chain_split<Tin, DKP>())
        return launch_wide_out<Tin, DKP, NP, NPP, 2>(p, st);
}
// Both chains of a backward pass side by side while they do not fill the SMs twice;
// beyond that one after the other: CTAs of both on an SM wait for instructions
// (6144 chunks of 64 x 64 heads: 3 of 10 cycles a warp waited, 366 us; in two launches, each with its own last
// wave, 292; in one launch with the reverse chains first 280).
template <typename Tin, int DKP>
cudaError_t launch_chain_both(const DeltaParams &p, cudaStream_t st)
{
    if (delta_wide(p, true))
        return launch_wide_each<Tin, DKP>(p, st);
    if constexpr (chain_split<Tin, DKP>())
        return launch_split_both<Tin, DKP>(p, st);
    else
        return launch_wide_both<Tin, DKP>(p, st);
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
