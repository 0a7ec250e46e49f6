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
// warps, and a chunk needs one barrier for its stage of shared memory.  The
// reverse pass has the same shape:
//     dV'^T = dO^T P + e^{c_last - c} (dS^T K^T),  dX^T = dV'^T T,  dR = -beta e^c dX,
//     dS^T <- e^{c_last} dS^T + (scale e^c dO)^T Q + dR^T K
// It needs nothing of the forward chain, so that a backward pass runs both in
// one launch.
// float16 K and Q are multiplied as they are, by scaled float16 parts.
//
// A long chain of few heads would leave most SMs idle (three heads of 65536 tokens:
// 1024 chunks one after the other, 4.2 ms).  Its chunks are cut into segments of SC.
// S -> M S + N over a segment, so a first pass runs every segment at once, from S = 0
// with its values for N and from S = 1 without values for M, delta_combine_kernel
// follows S over the segments, and the chain proper then runs every segment from its
// state.  The reverse chain's transition is M^T: its first pass adds only its own N.
//  A last chunk of up to
// 32 tokens is gone through as half a chunk.
#pragma once

#include "ss2d_delta.cuh"

namespace ss2d {

enum { kChainOut = 0, kChainState = 1, kChainRev = 2 };

template <typename Tin, int DKP, int NW, int MODE, int NP, int NPP, int STAGES>
struct ChainLayout {
    static constexpr int NPI = DeltaParts<Tin>::n;
    static constexpr bool HALF = std::is_same_v<Tin, __half>;    // K and Q as they are
    static constexpr int NKQ = HALF ? 1 : NPI;                   // their parts
    static constexpr int DVT = NW * 16;
    static constexpr int KB = NKQ * kDeltaC * DKP * 2;           // K; Q the same
    static constexpr int VRB = sizeof(Tin) == 2 ? DVT * 2 : (DVT + 4) * 4;   // row of V or dO
    static constexpr int oK = 0;
    static constexpr int oQ = KB;
    static constexpr int oV = MODE == kChainState ? oQ : oQ + KB;
    static constexpr int oT = oV + kDeltaC * VRB;
    static constexpr int oP = oT + NP * kTriBytes;
    static constexpr int oX = MODE == kChainState ? oP : oP + NPP * kTriBytes;   // e^c, e^{c_last - c}, beta
    static constexpr int stage = (oX + 3 * kDeltaC * 4 + 127) / 128 * 128;
    static constexpr int out = sizeof(Tin) == 2 && MODE != kChainState ? NW * kDeltaC * 32 : 0;
    static constexpr int bytes = STAGES * stage + out;
};

// NP parts of intermediate values (states, X, V'), NPP of P and of what only the
// output is made of.  tile: the block's tile of DV, or of DK for a segment's transition
// (ident).  LOCAL: the first pass over a segment, which only leaves its end; every: also
// of the segment that no other follows
template <typename Tin, int DKP, int NW, int MODE, int NP, int NPP, int STAGES, bool LOCAL>
__device__ __forceinline__ void delta_chain(const DeltaParams &p, int tile, bool ident, long long units,
                                            bool every = false, unsigned z0 = blockIdx.z, unsigned zn = gridDim.z)
{
    using Lay = ChainLayout<Tin, DKP, NW, MODE, NP, NPP, STAGES>;
    constexpr bool HALF = Lay::HALF;
    constexpr int NPI = Lay::NPI, NKQ = Lay::NKQ, NT = NW * 32, RBK = DKP * 2, PBK = kDeltaC * RBK, NK = DKP / 8;
    extern __shared__ __align__(128) unsigned char dsm[];
    const uint32_t sm0 = smem_addr(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t2 = (lane & 3) * 2;   // row and first column of a lane in an accumulator tile
    const int h = blockIdx.y, hk = h / (p.H / p.HK);
    const int dvw = (tile * NW + warp) * 16;   // first of the warp's DV columns
    const bool won = dvw < (LOCAL && ident ? p.DK : p.DV);
    __shared__ int ranked;
    for (long long z = z0; z < units; z += zn) {
        // packed sequences are taken by length, the longest first: the last chains to start are short ones
        long long unit = z;
        if (p.cu && !p.SC && p.nseq <= NT) {
            if (tid < p.nseq) {
                const int len = delta_seq(p, tid).len;
                int before = 0;
                for (int i = 0; i < p.nseq; ++i) {
                    const int l = delta_seq(p, i).len;
                    before += l > len || (l == len && i < tid);
                }
                if (before == (int)z)
                    ranked = tid;
            }
            __syncthreads();
            unit = ranked;
        }
        int sn, c0, c1;
        DeltaSeq q;
        if (!delta_unit(p, unit, sn, q, c0, c1))
            continue;
        const long long slot0 = delta_slot0(p, sn, q), su = unit * p.H + h;
        const int nchunks = (q.len + kDeltaC - 1) / kDeltaC, nc = c1 - c0;
        if (LOCAL && !every && (MODE == kChainRev ? c0 == 0 : c1 == nchunks))
            continue;
        auto chunk = [&](int i) { return MODE == kChainRev ? c1 - 1 - i : c0 + i; };

        // copies chunk c's operands into stage st
        auto load = [&](int c, int st) {
            const uint32_t base = sm0 + st * Lay::stage;
            const long long slot = slot0 + c, sh = slot * p.H + h;
            const int t0 = c * kDeltaC;
            for (int i = tid; i < NKQ * kDeltaC * (DKP / 8); i += NT) {
                const int r = i / (DKP / 8), pc = i % (DKP / 8);   // r counts the parts' rows
                const uint32_t dst = base + (r / kDeltaC) * PBK + swz<RBK>(r % kDeltaC, pc);
                const char *ks, *qs;
                bool on = true;
                if constexpr (NKQ == 1) {
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
            for (int i = tid; i < NP * kTriBytes / 16; i += NT)
                cp16(base + Lay::oT + i * 16, static_cast<const char *>(p.Tp) + sh * NP * kTriBytes + i * 16, true);
            if constexpr (MODE != kChainState)
                for (int i = tid; i < NPP * kTriBytes / 16; i += NT)
                    cp16(base + Lay::oP + i * 16, static_cast<const char *>(p.Pp) + sh * NPP * kTriBytes + i * 16,
                         true);
            constexpr int VPC = Lay::DVT * (int)sizeof(Tin) / 16, VPE = 16 / (int)sizeof(Tin);
            for (int i = tid; i < (LOCAL && ident ? 0 : kDeltaC * VPC); i += NT) {
                const int r = i / VPC, pc = i % VPC, d = tile * Lay::DVT + pc * VPE;
                const bool on = t0 + r < q.len && d < p.DV;
                const long long tok = delta_token(p, q, on ? t0 + r : 0);
                const Tin *src = MODE == kChainRev ? static_cast<const Tin *>(p.dout) + (tok * p.H + h) * p.DV
                                                   : static_cast<const Tin *>(p.v) + tok * p.vs + (long long)h * p.DV;
                const uint32_t dst = sizeof(Tin) == 2 ? swz<Lay::DVT * 2>(r, pc) : (uint32_t)(r * Lay::VRB + pc * 16);
                cp16(base + Lay::oV + dst, src + (on ? d : 0), on);
            }
            if (tid < 3 * kDeltaC * 4 / 16)
                cp16(base + Lay::oX + tid * 16, p.vec + sh * kDeltaVec + tid * 4, true);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };
        // V or dO of the warp's columns and 16 tokens, transposed, in accumulator layout
        auto values = [&](const unsigned char *base, int blk, float (&v0)[4], float (&v1)[4]) {
            if constexpr (sizeof(Tin) == 2) {
                uint32_t r[4];
                ldsm4t(smem_addr(base) + Lay::oV +
                           swz<Lay::DVT * 2>(blk * 16 + (lane & 7) + (lane >> 4) * 8, warp * 2 + (lane >> 3 & 1)),
                       r);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v0[j * 2] = half_bits_to_f32<Tin>(r[j] & 0xffffu);
                    v0[j * 2 + 1] = half_bits_to_f32<Tin>(r[j] >> 16);
                    v1[j * 2] = half_bits_to_f32<Tin>(r[2 + j] & 0xffffu);
                    v1[j * 2 + 1] = half_bits_to_f32<Tin>(r[2 + j] >> 16);
                }
            } else {
                const float *vt = reinterpret_cast<const float *>(base + Lay::oV) + warp * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v0[j] = vt[(blk * 16 + t2 + (j & 1)) * (Lay::DVT + 4) + g8 + (j >> 1) * 8];
                    v1[j] = vt[(blk * 16 + 8 + t2 + (j & 1)) * (Lay::DVT + 4) + g8 + (j >> 1) * 8];
                }
            }
        };
        // a 16 x 64 result, transposed back and rounded, into the rows of a (tokens, H, DV) tensor
        auto emit = [&](const float (&v)[8][4], void *dst, int t0) {
            if constexpr (sizeof(Tin) == 2) {
                const uint32_t ob = sm0 + STAGES * Lay::stage + warp * kDeltaC * 32;
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
                        const uint4 u = *reinterpret_cast<const uint4 *>(dsm + STAGES * Lay::stage +
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
            const float *sin = (MODE == kChainRev ? p.dSin : p.Sin) + (su * p.DV + dvw + g8) * DKP;
#pragma unroll
            for (int n = 0; n < NK; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int dk = n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                    if constexpr (LOCAL)
                        S[n][j] = ident && dk == dv && dk < p.DK ? 1.f : 0.f;
                    else if (p.SC)
                        S[n][j] = won ? sin[(j >> 1) * 8 * DKP + dk] : 0.f;
                    else
                        S[n][j] = src && won && dk < p.DK
                                      ? src[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv]
                                      : 0.f;
                }
        }
        if (nc > 0)
            load(chunk(0), 0);
        for (int i = 0; i < nc; ++i) {
            const int c = chunk(i), st = STAGES == 2 ? i & 1 : 0, t0 = c * kDeltaC;
            const long long sh = (slot0 + c) * p.H + h;
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");
            __syncthreads();   // the stage is here, and every warp is done with the other one
            if (STAGES == 2 && i + 1 < nc)
                load(chunk(i + 1), st ^ 1);
            const unsigned char *sb = dsm + st * Lay::stage;
            const uint32_t sa = sm0 + st * Lay::stage;
            const float *eg = reinterpret_cast<const float *>(sb + Lay::oX), *el = eg + kDeltaC, *be = el + kDeltaC;
            // NB: blocks of 16 tokens gone through, all four or the first two.  Unrolled without branches, the
            // products of neighbouring blocks overlap; with a test before each block the chain of one sequence
            // took 5.9 us a chunk instead of 4.1.
            auto step = [&](auto blocks) {
                constexpr int NB = decltype(blocks)::value;
                if constexpr (MODE != kChainOut && !LOCAL) {
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
                // (K S)^T
                [[maybe_unused]] HalfScale hs{{1.f, 1.f}, {1.f, 1.f}};
                if constexpr (HALF)
                    hs = half_scale(S);
#pragma unroll
                for (int ks = 0; ks < DKP / 16; ++ks) {
                    if constexpr (HALF) {
                        uint32_t a[2][4], kb[1][4];
                        half_frag(S[2 * ks], S[2 * ks + 1], hs.up, a);
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b < NB) {
                                frag_rows<RBK, 1>(sa + Lay::oK, PBK, b * 16, ks * 2, kb);
                                mma_half<NP == 3>(R[2 * b], R[2 * b + 1], a, kb[0], hs.down);
                            }
                    } else {
                        uint32_t a[NP][4];
                        frag_a<NP>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b < NB)
                                mma_rows<RBK, NP, NPI, NP>(R[2 * b], R[2 * b + 1], a, sa + Lay::oK, PBK, b * 16,
                                                           ks * 2);
                    }
                }
                if constexpr (HALF && NP != 3) {
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[n][j] *= hs.down[j >> 1];
                }
                if constexpr (MODE != kChainRev) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (b < NB) {
                            float v[2][4] = {};
                            if (!(LOCAL && ident))
                                values(sb, b, v[0], v[1]);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    R[2 * b + e][j] = v[e][j] - eg[b * 16 + e * 8 + t2 + (j & 1)] * R[2 * b + e][j];
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                R[2 * b + e][j] *= be[b * 16 + e * 8 + t2 + (j & 1)];   // X
                    }
                    // V'^T = X^T T^T
                    float W[8][4];
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            W[n][j] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (ks >= NB)
                            continue;
                        uint32_t a[NP][4];
                        frag_a<NP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                        for (int b = ks; b < 4; ++b)
                            if (b < NB)
                                mma_block_rows<NP, NP, NP>(W[2 * b], W[2 * b + 1], a,
                                                           sa + Lay::oT + tri_block(b, ks));
                    }
                    if constexpr (MODE == kChainOut) {
                        // O^T = scale e^c (Q S)^T + V'^T P^T
#pragma unroll
                        for (int ks = 0; ks < DKP / 16; ++ks) {
                            if constexpr (HALF) {
                                uint32_t a[2][4], qb[1][4];
                                half_frag(S[2 * ks], S[2 * ks + 1], hs.up, a);
#pragma unroll
                                for (int b = 0; b < 4; ++b)
                                    if (b < NB) {
                                        frag_rows<RBK, 1>(sa + Lay::oQ, PBK, b * 16, ks * 2, qb);
                                        mma_half<false>(O[2 * b], O[2 * b + 1], a, qb[0], hs.down);
                                    }
                            } else {
                                uint32_t a[NPP][4];
                                frag_a<NPP>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
                                for (int b = 0; b < 4; ++b)
                                    if (b < NB)
                                        mma_rows<RBK, NPP, NPI, NPP>(O[2 * b], O[2 * b + 1], a, sa + Lay::oQ, PBK,
                                                                     b * 16, ks * 2);
                            }
                        }
                        const float os[2] = {p.scale * (HALF ? hs.down[0] : 1.f), p.scale * (HALF ? hs.down[1] : 1.f)};
#pragma unroll
                        for (int n = 0; n < 8; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                O[n][j] *= os[j >> 1] * eg[n * 8 + t2 + (j & 1)];
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            if (ks >= NB)
                                continue;
                            uint32_t a[NPP][4];
                            frag_a<NPP>(W[2 * ks], W[2 * ks + 1], a);
#pragma unroll
                            for (int b = ks; b < 4; ++b)
                                if (b < NB)
                                    mma_block_rows<NPP, NPP, NPP>(O[2 * b], O[2 * b + 1], a,
                                                                  sa + Lay::oP + tri_block(b, ks));
                        }
                        emit(O, p.o, t0);
                    } else if constexpr (!LOCAL) {
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            put(p.Vx, sh, kDeltaC, n, W[n]);
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[n][j] = W[n][j] * el[n * 8 + t2 + (j & 1)];
                } else {
                    // dV'^T = dO^T P + e^{c_last - c} (K dS)^T: row i of P holds its columns j <= i
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[n][j] *= el[n * 8 + t2 + (j & 1)];
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (ks >= NB)
                            continue;
                        float v[2][4];
                        values(sb, ks, v[0], v[1]);
                        uint32_t a[NPI][4];
                        frag_a<NPI>(v[0], v[1], a);
#pragma unroll
                        for (int b = 0; b <= ks; ++b)
                            mma_block_cols<NPI, NPP, NPP>(R[2 * b], R[2 * b + 1], a,
                                                          sa + Lay::oP + tri_block(ks, b));
                    }
                    // dX^T = dV'^T T
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (ks >= NB)
                            continue;
                        uint32_t a[NP][4];
                        frag_a<NP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                        for (int b = 0; b <= ks; ++b)
                            mma_block_cols<NP, NP, NP>(O[2 * b], O[2 * b + 1], a, sa + Lay::oT + tri_block(ks, b));
                    }
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        if constexpr (!LOCAL)
                            put(p.dXx, sh, kDeltaC, n, O[n]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            O[n][j] *= be[n * 8 + t2 + (j & 1)];
                            R[n][j] = -eg[n * 8 + t2 + (j & 1)] * O[n][j];   // dR
                        }
                    }
                    if constexpr (!LOCAL)
                        emit(O, p.dv, t0);
                }
                // S^T <- e^{c_last} S^T + (e^{c_last - c} V')^T K, or dR^T K + (scale e^c dO)^T Q
                const float elast = eg[kDeltaC - 1];
#pragma unroll
                for (int n = 0; n < NK; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[n][j] *= elast;
                if constexpr (HALF)
                    hs = half_scale(R);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    if (ks >= NB)
                        continue;
                    // S^T += A B in two float16 parts of A
                    auto half_cols = [&](const float (&c0)[4], const float (&c1)[4], const HalfScale &h, int at) {
                        uint32_t a[2][4], kb[1][4];
                        half_frag(c0, c1, h.up, a);
#pragma unroll
                        for (int nt = 0; nt < NK; nt += 2) {
                            frag_cols<RBK, 1>(sa + at, PBK, ks * 16, nt, kb);
                            mma_half<true>(S[nt], S[nt + 1], a, kb[0], h.down);
                        }
                    };
                    [[maybe_unused]] uint32_t a[NP][4];
                    if constexpr (HALF) {
                        half_cols(R[2 * ks], R[2 * ks + 1], hs, Lay::oK);
                    } else {
                        frag_a<NP>(R[2 * ks], R[2 * ks + 1], a);
#pragma unroll
                        for (int nt = 0; nt < NK; nt += 2)
                            mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sa + Lay::oK, PBK, ks * 16, nt);
                    }
                    if constexpr (MODE == kChainRev) {
                        float v[2][4];
                        values(sb, ks, v[0], v[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[e][j] *= p.scale * eg[ks * 16 + e * 8 + t2 + (j & 1)];
                        if constexpr (HALF) {
                            half_cols(v[0], v[1], half_scale(v), Lay::oQ);
                        } else {
                            frag_a<NP>(v[0], v[1], a);
#pragma unroll
                            for (int nt = 0; nt < NK; nt += 2)
                                mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sa + Lay::oQ, PBK, ks * 16, nt);
                        }
                    }
                }
            };
            if (won) {
                if (q.len - t0 > 32)
                    step(std::integral_constant<int, 4>());
                else
                    step(std::integral_constant<int, 2>());
            }
            if (STAGES == 1 && i + 1 < nc) {
                __syncthreads();
                load(chunk(i + 1), 0);
            }
        }
        if constexpr (LOCAL) {
            if (won && ident) {
                uint32_t *m = static_cast<uint32_t *>(p.Ms);
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    uint32_t w[3], u[3];
                    split2<3>(S[n][0], S[n][1], w);
                    split2<3>(S[n][2], S[n][3], u);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        uint32_t *r = m + (((su * 3 + k) * DKP + dvw + g8) * DKP + n * 8 + t2) / 2;
                        r[0] = w[k];
                        r[8 * DKP / 2] = u[k];
                    }
                }
            } else if (won) {
#pragma unroll
                for (int n = 0; n < NK; ++n)
                    put(MODE == kChainRev ? p.dNs : p.Ns, su, DKP, n, S[n]);
            }
        } else {
            float *dst = MODE == kChainRev ? p.dh0 : p.h_last;
            if (dst && won && (MODE == kChainRev ? c0 == 0 : c1 == nchunks)) {
#pragma unroll
                for (int n = 0; n < NK; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int dk = n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                        if (dk < p.DK)
                            dst[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv] = S[n][j];
                    }
            }
        }
        __syncthreads();
    }
}

// CTAs per SM that the registers are held to: three of four warps where three stages of shared memory fit and
// 168 registers do (not the output's chain with three parts: 328 bytes of spills)
template <typename Lay, int DKP, int STAGES, bool OUT3 = false>
constexpr int chain_ctas() { return STAGES == 1 && DKP == 64 && Lay::bytes <= 74 * 1024 && !OUT3 ? 3 : 2; }

template <typename Tin, int DKP, int NW, int NP, int NPP, int STAGES>
__global__ void
    __launch_bounds__(NW * 32,
                      (chain_ctas<ChainLayout<Tin, DKP, NW, kChainOut, NP, NPP, STAGES>, DKP, STAGES, NP == 3>()))
        delta_out_kernel(const DeltaParams p, long long units)
{
    delta_chain<Tin, DKP, NW, kChainOut, NP, NPP, STAGES, false>(p, blockIdx.x, false, units);
}
// all reverse chains, then all forward ones (the second half of blockIdx.z)
template <typename Tin, int DKP, int NW, int STAGES>
__global__ void
    __launch_bounds__(NW * 32, (chain_ctas<ChainLayout<Tin, DKP, NW, kChainRev, 3, 3, STAGES>, DKP, STAGES>()))
        delta_each_kernel(const DeltaParams p, long long units)
{
    const unsigned zn = gridDim.z / 2;
    if (blockIdx.z < zn)
        delta_chain<Tin, DKP, NW, kChainRev, 3, 3, STAGES, false>(p, blockIdx.x, false, units, false, blockIdx.z, zn);
    else
        delta_chain<Tin, DKP, NW, kChainState, 3, 3, STAGES, false>(p, blockIdx.x, false, units, false,
                                                                     blockIdx.z - zn, zn);
}
// the forward chain and the reverse one side by side, the longer one first
template <typename Tin, int DKP, int NW, int STAGES>
__global__ void __launch_bounds__(NW * 32,
                                  (chain_ctas<ChainLayout<Tin, DKP, NW, kChainRev, 3, 3, STAGES>, DKP, STAGES>()))
    delta_both_kernel(const DeltaParams p, long long units)
{
    if (blockIdx.x & 1)
        delta_chain<Tin, DKP, NW, kChainState, 3, 3, STAGES, false>(p, blockIdx.x >> 1, false, units);
    else
        delta_chain<Tin, DKP, NW, kChainRev, 3, 3, STAGES, false>(p, blockIdx.x >> 1, false, units);
}

// first pass over the segments: tiles of DV forward, of DK for the transition, and of DV in reverse (REV)
template <typename Tin, int DKP, int NP, int STAGES, bool REV>
__global__ void __launch_bounds__(128, 2) delta_local_kernel(const DeltaParams p, int dvt, int dkt, long long units)
{
    const int x = blockIdx.x;
    if (x < dvt + dkt)
        delta_chain<Tin, DKP, 4, kChainState, NP, 3, STAGES, true>(p, x < dvt ? x : x - dvt, x >= dvt, units,
                                                                     REV && x >= dvt);
    else if constexpr (REV)
        delta_chain<Tin, DKP, 4, kChainRev, NP, 3, STAGES, true>(p, x - dvt - dkt, false, units);
}

// The states that the segments of a sequence start from (blockIdx.x even: dS that
// they end with): S <- M S + N over them, transposed, 16 columns of DV to a CTA, a
// warp 16 of the result's columns.  One step is DKP^2 products of three parts a column;
// a warp leaves the parts of its columns in shared memory, where all read the next
// step's A operand.  The next transitions are copied meanwhile.  Steps follow one
// another, so they are spread over SMs: with 64 columns of DV to a CTA and S kept in
// a warp's registers a step of 64 x 64 took 2.3 us.  Sequences of no tokens pass their
// state on.
template <int DKP>
struct CombineLayout {
    static constexpr int stages = DKP == 64 ? 4 : 2;
    static constexpr int RB = DKP * 2, PB = DKP * RB, STG = 3 * PB;   // a row, a part, a transition
    static constexpr int SP = 16 * RB;                       // one part of S^T
    static constexpr int oS = stages * STG;                  // two buffers of S^T
    static constexpr int bytes = oS + 2 * 3 * SP;
    static constexpr int threads = DKP * 2;
};

template <int DKP, bool REV>
__global__ void __launch_bounds__(CombineLayout<DKP>::threads) delta_combine_kernel(const DeltaParams p)
{
    using Lay = CombineLayout<DKP>;
    constexpr int RB = Lay::RB, PB = Lay::PB, STG = Lay::STG, STAGES = Lay::stages, NH = 2;
    extern __shared__ __align__(128) unsigned char dsm[];
    const uint32_t sa = smem_addr(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t2 = (lane & 3) * 2;
    const int h = blockIdx.y, tile = REV ? blockIdx.x >> 1 : blockIdx.x;
    const bool rev = REV && !(blockIdx.x & 1);
    const int dvw = tile * 16, dk0 = warp * 16;
    for (int sn = blockIdx.z; sn < p.nseq; sn += gridDim.z) {
        const DeltaSeq q = delta_seq(p, sn);
        const int nc = (q.len + kDeltaC - 1) / kDeltaC, ns = (nc + p.SC - 1) / p.SC;
        const long long u0 = delta_seg0(p, sn, q);
        auto seg = [&](int i) { return (u0 + (rev ? ns - 1 - i : i)) * p.H + h; };
        auto load = [&](int i) {
            const char *src = static_cast<const char *>(p.Ms) + seg(i) * STG;
            for (int k = tid; k < STG / 16; k += Lay::threads) {
                const int r = k / (DKP / 8), pc = k % (DKP / 8);   // r counts the parts' rows
                cp16(sa + i % STAGES * STG + r / DKP * PB + swz<RB>(r % DKP, pc), src + (long long)k * 16,
                     r % DKP < p.DK);
            }
        };
        const float *src = rev ? p.dh_last : p.h0;
        float S[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int dk = dk0 + n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                S[n][j] =
                    src && dk < p.DK ? src[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv] : 0.f;
            }
        // one group of copies for each step, empty past the end
        for (int i = 0; i < STAGES - 1; ++i) {
            if (i + 1 < ns)
                load(i);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        }
        for (int i = 0; i < ns; ++i) {
            const long long o = (seg(i) * p.DV + dvw + g8) * DKP + dk0 + t2;
            float A[NH][4];
            const int sbuf = Lay::oS + (i & 1) * 3 * Lay::SP;
            {
                float *dst = (rev ? p.dSin : p.Sin) + o;
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(S[n][0], S[n][1]);
                    *reinterpret_cast<float2 *>(dst + 8 * DKP + n * 8) = make_float2(S[n][2], S[n][3]);
                }
            }
            if (i + 1 == ns)
                break;
            {
                const float *N = (rev ? p.dNs : p.Ns) + o;
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    const float2 a = *reinterpret_cast<const float2 *>(N + n * 8);
                    const float2 b = *reinterpret_cast<const float2 *>(N + 8 * DKP + n * 8);
                    A[n][0] = a.x;
                    A[n][1] = a.y;
                    A[n][2] = b.x;
                    A[n][3] = b.y;
                }
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[3];
                        split2<3>(S[n][2 * e], S[n][2 * e + 1], w);
#pragma unroll
                        for (int m = 0; m < 3; ++m)
                            *reinterpret_cast<uint32_t *>(dsm + sbuf + m * Lay::SP +
                                                          swz<RB>(g8 + 8 * e, warp * 2 + n) + t2 * 2) = w[m];
                    }
            }
            asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 2) : "memory");
            __syncthreads();   // the transition and S are here, the last step's stage is read
            if (i + STAGES < ns)
                load(i + STAGES - 1);
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            {
                const uint32_t m = sa + i % STAGES * STG;
#pragma unroll
                for (int ks = 0; ks < DKP / 16; ++ks) {
                    uint32_t a[3][4];
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        ldsm4(sa + sbuf + k * Lay::SP + swz<RB>(lane & 15, ks * 2 + (lane >> 4)), a[k]);
#pragma unroll
                    for (int nt = 0; nt < NH; nt += 2) {
                        if (rev)
                            mma_rows<RB, 3, 3, 3>(A[nt], A[nt + 1], a, m, PB, dk0 + nt * 8, ks * 2);
                        else
                            mma_cols<RB, 3, 3, 3>(A[nt], A[nt + 1], a, m, PB, ks * 16, warp * 2 + nt);
                    }
                }
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[n][j] = A[n][j];
            }
        }
        float *dst = rev ? p.dh0 : p.h_last;
        if (ns == 0 && dst) {
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int dk = dk0 + n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                    if (dk < p.DK)
                        dst[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv] = S[n][j];
                }
        }
        cp_wait();
        __syncthreads();
    }
}

}  // namespace ss2d
