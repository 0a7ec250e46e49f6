// ss2d_delta_chain.cuh -- the chain of a sequence's states over its chunks,
// forward (outputs and last state, or the states and V' that a backward pass
// needs) and in reverse (the gradient of the states).
//
// Everything is computed transposed, with DV along the rows: a warp owns 16
// columns of DV and holds their S^T (16 x DK) in float32 accumulators. Then
//     (K S)^T = S^T K^T,  V'^T = X^T T^T,  O^T = S^T Q^T + V'^T P^T,
//     S^T <- e^{c_last} S^T + (e^{c_last - c} V')^T K
// have as A operand what the warp just computed (an accumulator fragment,
// split into bf16 parts, is an A fragment lane by lane) and as B operand K, Q,
// T or P from shared memory, by rows or by columns.  No value passes between
// warps, and a chunk needs one barrier, for the stage of shared memory that
// the next chunk is copied into meanwhile.  The reverse pass has the same
// shape:
//     dV'^T = dO^T P + e^{c_last - c} (dS^T K^T),  dX^T = dV'^T T,  dR = -beta e^c dX,
//     dS^T <- e^{c_last} dS^T + (scale e^c dO)^T Q + dR^T K
// T and P are lower triangular in 16 x 16 blocks: the blocks above the
// diagonal are neither copied nor multiplied.
#pragma once

#include "ss2d_delta.cuh"

namespace ss2d {

enum { kChainOut = 0, kChainState = 1, kChainRev = 2 };

template <typename Tin, int DKP, int NW, int MODE, int NP, int NPP>
struct ChainLayout {
    static constexpr int NPI = DeltaParts<Tin>::n;
    static constexpr int DVT = NW * 16;
    static constexpr int KB = NPI * kDeltaC * DKP * 2;           // K; Q the same
    static constexpr int TB = kDeltaC * kDeltaC * 2;             // one part of T or P
    static constexpr int VRB = sizeof(Tin) == 2 ? DVT * 2 : (DVT + 4) * 4;   // row of V or dO
    static constexpr int oK = 0;
    static constexpr int oQ = KB;
    static constexpr int oT = MODE == kChainState ? oQ : oQ + KB;
    static constexpr int oP = oT + NP * TB;
    static constexpr int oV = MODE == kChainState ? oP : oP + NPP * TB;
    static constexpr int oX = oV + kDeltaC * VRB;                // e^c, e^{c_last - c}, beta
    static constexpr int stage = (oX + 3 * kDeltaC * 4 + 127) / 128 * 128;
    static constexpr int out = sizeof(Tin) == 2 && MODE != kChainState ? NW * kDeltaC * 32 : 0;
    static constexpr int stages = 2 * stage + out <= 225 * 1024 ? 2 : 1;
    static constexpr int bytes = stages * stage + out;
};

// NP parts of intermediate values (states, X, V'), NPP of P and of what only the output is made of
template <typename Tin, int DKP, int NW, int MODE, int NP, int NPP>
__global__ void __launch_bounds__(NW * 32, 1) delta_chain_kernel(const DeltaParams p)
{
    using Lay = ChainLayout<Tin, DKP, NW, MODE, NP, NPP>;
    constexpr int NPI = Lay::NPI, NT = NW * 32, RBK = DKP * 2, PBK = kDeltaC * RBK, NK = DKP / 8;
    extern __shared__ __align__(128) unsigned char dsm[];
    const uint32_t sm0 = smem_addr(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t2 = (lane & 3) * 2;   // row and first column of a lane in an accumulator tile
    const int h = blockIdx.y, hk = h / (p.H / p.HK);
    const int dvw = (blockIdx.x * NW + warp) * 16;   // first of the warp's DV columns
    const bool won = dvw < p.DV;
    for (int sn = blockIdx.z; sn < p.nseq; sn += gridDim.z) {
        const DeltaSeq q = delta_seq(p, sn);
        const int nc = (q.len + kDeltaC - 1) / kDeltaC;
        const long long slot0 = delta_slot0(p, sn, q);
        auto chunk = [&](int i) { return MODE == kChainRev ? nc - 1 - i : i; };

        // copies chunk c's operands into stage st
        auto load = [&](int c, int st) {
            const uint32_t base = sm0 + st * Lay::stage;
            const long long slot = slot0 + c, sh = slot * p.H + h;
            const int t0 = c * kDeltaC;
            for (int i = tid; i < NPI * kDeltaC * (DKP / 8); i += NT) {
                const int r = i / (DKP / 8), pc = i % (DKP / 8);   // r counts the parts' rows
                const uint32_t dst = base + (r / kDeltaC) * PBK + swz<RBK>(r % kDeltaC, pc);
                const char *ks, *qs;
                bool on = true;
                if constexpr (NPI == 1) {
                    on = t0 + r < q.len && pc * 8 < p.DK;
                    const long long tok = delta_token(p, q, on ? t0 + r : 0);
                    const long long col = (long long)hk * p.DK + (on ? pc * 8 : 0);
                    ks = static_cast<const char *>(p.k) + (tok * p.ks + col) * 2;
                    qs = static_cast<const char *>(p.q) + (tok * p.qs + col) * 2;
                } else {
                    const long long o = (slot * p.HK + hk) * (NPI * PBK) + (long long)i * 16;
                    ks = static_cast<const char *>(p.kp) + o;
                    qs = static_cast<const char *>(p.qp) + o;
                }
                cp16(dst + Lay::oK, ks, on);
                if constexpr (MODE != kChainState)
                    cp16(dst + Lay::oQ, qs, on);
            }
            for (int i = tid; i < kDeltaC * 8; i += NT) {
                const int r = i >> 3, pc = i & 7;
                if (pc / 2 > r / 16)
                    continue;
#pragma unroll
                for (int m = 0; m < NP; ++m)
                    cp16(base + Lay::oT + m * Lay::TB + swz<128>(r, pc),
                         static_cast<const char *>(p.Tp) + (sh * NP + m) * Lay::TB + i * 16, true);
                if constexpr (MODE != kChainState) {
#pragma unroll
                    for (int m = 0; m < NPP; ++m)
                        cp16(base + Lay::oP + m * Lay::TB + swz<128>(r, pc),
                             static_cast<const char *>(p.Pp) + (sh * NPP + m) * Lay::TB + i * 16, true);
                }
            }
            constexpr int VPC = Lay::DVT * (int)sizeof(Tin) / 16, VPE = 16 / (int)sizeof(Tin);
            for (int i = tid; i < kDeltaC * VPC; i += NT) {
                const int r = i / VPC, pc = i % VPC, d = blockIdx.x * Lay::DVT + pc * VPE;
                const bool on = t0 + r < q.len && d < p.DV;
                const long long tok = delta_token(p, q, on ? t0 + r : 0);
                const Tin *src = MODE == kChainRev ? static_cast<const Tin *>(p.dout) + (tok * p.H + h) * p.DV
                                                   : static_cast<const Tin *>(p.v) + tok * p.vs + (long long)h * p.DV;
                const uint32_t dst = sizeof(Tin) == 2 ? swz<Lay::DVT * 2>(r, pc) : (uint32_t)(r * Lay::VRB + pc * 16);
                cp16(base + Lay::oV + dst, src + (on ? d : 0), on);
            }
            if (tid < 3 * kDeltaC * 4 / 16)
                cp16(base + Lay::oX + tid * 16, p.vec + sh * 3 * kDeltaC + tid * 4, true);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };
        // V or dO of the warp's columns, transposed, in accumulator layout
        auto values = [&](const unsigned char *base, float (&v)[8][4]) {
            if constexpr (sizeof(Tin) == 2) {
#pragma unroll
                for (int nt = 0; nt < 8; nt += 2) {
                    uint32_t r[4];
                    ldsm4t(smem_addr(base) + Lay::oV +
                               swz<Lay::DVT * 2>(nt * 8 + (lane & 7) + (lane >> 4) * 8, warp * 2 + (lane >> 3 & 1)),
                           r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[nt + (j >> 1)][(j & 1) * 2] = half_bits_to_f32<Tin>(r[j] & 0xffffu);
                        v[nt + (j >> 1)][(j & 1) * 2 + 1] = half_bits_to_f32<Tin>(r[j] >> 16);
                    }
                }
            } else {
                const float *vt = reinterpret_cast<const float *>(base + Lay::oV) + warp * 16;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[nt][j] = vt[(nt * 8 + t2 + (j & 1)) * (Lay::DVT + 4) + g8 + (j >> 1) * 8];
            }
        };
        // a 16 x 64 result, transposed back and rounded, into the rows of a (tokens, H, DV) tensor
        auto emit = [&](const float (&v)[8][4], void *dst, int t0) {
            if constexpr (sizeof(Tin) == 2) {
                const uint32_t ob = sm0 + Lay::stages * Lay::stage + warp * kDeltaC * 32;
#pragma unroll
                for (int nt = 0; nt < 8; nt += 2) {
                    uint32_t r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a = v[nt + (j >> 1)][(j & 1) * 2], b = v[nt + (j >> 1)][(j & 1) * 2 + 1];
                        if constexpr (std::is_same_v<Tin, __half>) {
                            const __half2 hh = __floats2half2_rn(a, b);
                            r[j] = *reinterpret_cast<const uint32_t *>(&hh);
                        } else {
                            r[j] = pack_bf16(a, b);
                        }
                    }
                    stsm4t(ob + (nt * 8 + (lane & 7) + (lane >> 4) * 8) * 32 + (lane >> 3 & 1) * 16, r);
                }
                __syncwarp();
#pragma unroll
                for (int i = lane; i < kDeltaC * 2; i += 32) {
                    const int t = t0 + (i >> 1);
                    if (won && t < q.len) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(dsm + Lay::stages * Lay::stage +
                                                                         warp * kDeltaC * 32 + i * 16);
                        *reinterpret_cast<uint4 *>(static_cast<Tin *>(dst) +
                                                   (delta_token(p, q, t) * p.H + h) * p.DV + dvw + (i & 1) * 8) = u;
                    }
                }
                __syncwarp();
            } else {
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = t0 + nt * 8 + t2 + (j & 1);
                        if (won && t < q.len)
                            static_cast<Tin *>(dst)[(delta_token(p, q, t) * p.H + h) * p.DV + dvw + g8 +
                                                    (j >> 1) * 8] = v[nt][j];
                    }
            }
        };
        // float pairs of a transposed scratch tile [DV][W]
        auto put = [&](float *dst, long long sh, int W, int n, const float (&v)[4]) {
            float *r = dst + (sh * p.DV + dvw + g8) * W + n * 8 + t2;
            *reinterpret_cast<float2 *>(r) = make_float2(v[0], v[1]);
            *reinterpret_cast<float2 *>(r + 8 * W) = make_float2(v[2], v[3]);
        };

        float S[NK][4];
        {
            const float *src = MODE == kChainRev ? p.dh_last : p.h0;
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int dk = n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                    S[n][j] = src && won && dk < p.DK
                                  ? src[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv]
                                  : 0.f;
                }
        }
        if (nc > 0)
            load(chunk(0), 0);
        for (int i = 0; i < nc; ++i) {
            const int c = chunk(i), st = Lay::stages == 2 ? i & 1 : 0, t0 = c * kDeltaC;
            const long long sh = (slot0 + c) * p.H + h;
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
            __syncthreads();   // the stage is here, and every warp is done with the other one
            if (Lay::stages == 2 && i + 1 < nc)
                load(chunk(i + 1), st ^ 1);
            const unsigned char *sb = dsm + st * Lay::stage;
            const uint32_t sa = sm0 + st * Lay::stage;
            const float *eg = reinterpret_cast<const float *>(sb + Lay::oX), *el = eg + kDeltaC, *be = el + kDeltaC;
            const float elast = eg[kDeltaC - 1];
            if (won) {
                if constexpr (MODE != kChainOut) {
                    float *dst = MODE == kChainRev ? p.dSx : p.Sx;
#pragma unroll
                    for (int n = 0; n < NK; ++n)
                        put(dst, sh, DKP, n, S[n]);
                }
                float R[8][4], O[8][4];
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        R[n][j] = O[n][j] = 0.f;
                // (K S)^T, and (Q S)^T for the output
#pragma unroll
                for (int ks = 0; ks < DKP / 16; ++ks) {
                    uint32_t a[NP][4];
                    frag_a<NP>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
                    for (int nt = 0; nt < 8; nt += 2) {
                        mma_rows<RBK, NP, NPI, NP>(R[nt], R[nt + 1], a, sa + Lay::oK, PBK, nt * 8, ks * 2);
                        if constexpr (MODE == kChainOut)
                            mma_rows<RBK, NP, NPI, NPP>(O[nt], O[nt + 1], a, sa + Lay::oQ, PBK, nt * 8, ks * 2);
                    }
                }
                float V[8][4];
                if constexpr (MODE != kChainRev) {
                    values(sb, V);
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            V[n][j] -= eg[n * 8 + t2 + (j & 1)] * R[n][j];   // Y
                        if constexpr (MODE == kChainState)
                            put(p.Yx, sh, kDeltaC, n, V[n]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            V[n][j] *= be[n * 8 + t2 + (j & 1)];             // X
                            R[n][j] = 0.f;
                        }
                    }
                    // V'^T = X^T T^T
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        uint32_t a[NP][4];
                        frag_a<NP>(V[2 * ks], V[2 * ks + 1], a);
#pragma unroll
                        for (int nt = 2 * ks; nt < 8; nt += 2)
                            mma_rows<128, NP, NP, NP>(R[nt], R[nt + 1], a, sa + Lay::oT, Lay::TB, nt * 8, ks * 2);
                    }
                    if constexpr (MODE == kChainOut) {
#pragma unroll
                        for (int n = 0; n < 8; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                O[n][j] *= p.scale * eg[n * 8 + t2 + (j & 1)];
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            uint32_t a[NPP][4];
                            frag_a<NPP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                            for (int nt = 2 * ks; nt < 8; nt += 2)
                                mma_rows<128, NPP, NPP, NPP>(O[nt], O[nt + 1], a, sa + Lay::oP, Lay::TB, nt * 8,
                                                             ks * 2);
                        }
                        emit(O, p.o, t0);
                    } else {
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            put(p.Vx, sh, kDeltaC, n, R[n]);
                    }
                    // S^T <- e^{c_last} S^T + (e^{c_last - c} V')^T K
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[n][j] *= el[n * 8 + t2 + (j & 1)];
                } else {
                    // R = (K dS)^T: its product with V' goes to the gradient of the decays
                    float kl[8][2];
                    const float *vx = p.Vx + (sh * p.DV + dvw + g8) * kDeltaC + t2;
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float2 v0 = *reinterpret_cast<const float2 *>(vx + n * 8);
                        const float2 v1 = *reinterpret_cast<const float2 *>(vx + 8 * kDeltaC + n * 8);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[n][j] *= el[n * 8 + t2 + (j & 1)];
                        kl[n][0] = fmaf(R[n][0], v0.x, R[n][2] * v1.x);
                        kl[n][1] = fmaf(R[n][1], v0.y, R[n][3] * v1.y);
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            for (int m = 4; m < 32; m <<= 1)
                                kl[n][e] += __shfl_xor_sync(0xffffffffu, kl[n][e], m);
                        }
                    if (g8 == 0) {
                        float *dst = p.klx + (sh * (p.DV / 16) + dvw / 16) * kDeltaC + t2;
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(kl[n][0], kl[n][1]);
                    }
                    // dV'^T = dO^T P + e^{c_last - c} (K dS)^T: row i of P holds its columns j <= i
                    values(sb, V);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        uint32_t a[NPI][4];
                        frag_a<NPI>(V[2 * ks], V[2 * ks + 1], a);
#pragma unroll
                        for (int nt = 0; nt <= 2 * ks; nt += 2)
                            mma_cols<128, NPI, NPP, NPP>(R[nt], R[nt + 1], a, sa + Lay::oP, Lay::TB, ks * 16, nt);
                    }
                    // dX^T = dV'^T T
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        uint32_t a[NP][4];
                        frag_a<NP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                        for (int nt = 0; nt <= 2 * ks; nt += 2)
                            mma_cols<128, NP, NP, NP>(O[nt], O[nt + 1], a, sa + Lay::oT, Lay::TB, ks * 16, nt);
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        put(p.dXx, sh, kDeltaC, n, O[n]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            O[n][j] *= be[n * 8 + t2 + (j & 1)];
                            R[n][j] = -eg[n * 8 + t2 + (j & 1)] * O[n][j];   // dR
                            V[n][j] *= p.scale * eg[n * 8 + t2 + (j & 1)];
                        }
                    }
                    emit(O, p.dv, t0);
                }
#pragma unroll
                for (int n = 0; n < NK; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[n][j] *= elast;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    uint32_t a[NP][4];
                    frag_a<NP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                    for (int nt = 0; nt < NK; nt += 2)
                        mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sa + Lay::oK, PBK, ks * 16, nt);
                    if constexpr (MODE == kChainRev) {
                        frag_a<NP>(V[2 * ks], V[2 * ks + 1], a);
#pragma unroll
                        for (int nt = 0; nt < NK; nt += 2)
                            mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sa + Lay::oQ, PBK, ks * 16, nt);
                    }
                }
            }
            if (Lay::stages == 1 && i + 1 < nc) {
                __syncthreads();
                load(chunk(i + 1), 0);
            }
        }
        float *dst = MODE == kChainRev ? p.dh0 : p.h_last;
        if (dst && won) {
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int dk = n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                    if (dk < p.DK)
                        dst[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv] = S[n][j];
                }
        }
        __syncthreads();
    }
}

}  // namespace ss2d
