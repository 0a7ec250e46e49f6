// ss2d_delta_launch.h -- internal interface between the gated delta rule's C
// ABI (ss2d_delta.cu) and its kernels, one translation unit per input type.
#pragma once

#include <cuda_runtime.h>

#include "ss2d_delta.cuh"

namespace ss2d {

// Layout of a chunked call's scratch, per chunk slot and head.
struct DeltaPlan {
    int dkp;       // DK padded to 64 or 128
    int npi;       // bf16 parts of an input value
    int np, npp;   // parts of T, of P
};

// what: the recurrent kernel or the chunked forward
enum { kDeltaRecur = 0, kDeltaFwd = 1, kDeltaBwd = 2 };
cudaError_t launch_delta_bf16(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st);
cudaError_t launch_delta_f16(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st);
cudaError_t launch_delta_f32(const DeltaParams &p, const DeltaPlan &pl, int what, cudaStream_t st);
cudaError_t launch_delta_bwd_bf16(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st);
cudaError_t launch_delta_bwd_f16(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st);
cudaError_t launch_delta_bwd_f32(const DeltaParams &p, const DeltaPlan &pl, cudaStream_t st);

// CTAs of 64 columns of DV above which a chain counts as many (two to an SM)
constexpr long long kWideCtas = 2 * 148;

// chains of a pass: segments (every slot that may hold one), or sequences
inline long long delta_units(const DeltaParams &p)
{
    if (!p.SC)
        return p.nseq;
    return p.cu ? p.nslots / p.SC + p.nseq : (long long)p.nseq * ((p.NC + p.SC - 1) / p.SC);
}
inline long long delta_ctas(const DeltaParams &p) { return (long long)((p.DV + 63) / 64) * p.H * delta_units(p); }
inline bool delta_wide(const DeltaParams &p, bool bwd) { return delta_ctas(p) * (bwd ? 2 : 1) > kWideCtas; }
// float16 outputs by four warps to 16 columns: wide heads, and so few that two CTAs of 32 columns have an SM each
inline bool delta_split_f16(const DeltaParams &p) { return !p.SC && delta_ctas(p) * 2 <= 148; }

}  // namespace ss2d
