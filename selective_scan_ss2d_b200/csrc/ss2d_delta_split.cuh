// ss2d_delta_split.cuh -- the chain of ss2d_delta_chain.cuh with four warps to 16
// columns of DV instead of one, for calls of few chains.
//
// A warp of the one-warp form has its scheduler to itself and issues a chunk's
// products, splits and copies one after the other: 4 to 10 us a chunk, the tensor pipe
// a third busy.  Here a warp of a group of four has
//     one token block (16 tokens) of R, X, V' and the output (dV', dX in reverse), and
//     a quarter of DK of the group's state, in float32 accumulators,
// and what the others need of it as an A operand (the parts of S, X, V', e^{..} V') goes
// through shared memory, split once by its owner.  A chunk has three meetings of a group (four in
// reverse) and two of the CTA.
// Every scheduler has four warps to choose from, whose blocks are rotated from group to
// group, since T and P give a block between one and four products.
// K of the next chunk is copied during this one; Q, T, P and V of this chunk
// while R is computed.
#pragma once

#include "ss2d_delta_chain.cuh"

namespace ss2d {

template <typename Tin, int DKP, int GROUPS, int MODE, int NP, int NPP, int KBUF>
struct SplitLayout {
    static constexpr int NPI = DeltaParts<Tin>::n;
    static constexpr int threads = GROUPS * 128, DVT = GROUPS * 16;
    static constexpr int RBK = DKP * 2, KB = NPI * kDeltaC * RBK;
    static constexpr int VRB = sizeof(Tin) == 4 ? (DVT + 4) * 4 : DVT * 2 + 16;   // row of V or dO
    static constexpr int SP = 16 * RBK;                // one part of a group's S
    static constexpr int XP = 16 * 128;                // one part of a group's X, V', ..
    static constexpr int oK = 0;
    static constexpr int oVec = KBUF * KB;             // e^c, e^{c_last - c}, beta; two of them
    static constexpr int oQ = oVec + 2 * 768;
    static constexpr int oV = oQ + (MODE == kChainState ? 0 : KB);
    static constexpr int oT = oV + kDeltaC * VRB;
    static constexpr int oP = oT + NP * kTriBytes;
    static constexpr int oG = oP + (MODE == kChainState ? 0 : NPP * kTriBytes);
    static constexpr int gS = 0, gX = NP * SP, gU = gX + NP * XP, group = gU + NP * XP;
    static constexpr int oE = oG + GROUPS * group;     // a warp's 16 x 16 results on their way out
    static constexpr int bytes = oE + (sizeof(Tin) == 2 && MODE != kChainState ? GROUPS * 4 * 512 : 0);
};

template <typename Tin, int DKP, int GROUPS, int MODE, int NP, int NPP, int KBUF, bool LOCAL>
__device__ __forceinline__ void delta_split(const DeltaParams &p, int tile, bool ident, long long units,
                                            bool every = false)
{
    using Lay = SplitLayout<Tin, DKP, GROUPS, MODE, NP, NPP, KBUF>;
    constexpr int NPI = Lay::NPI, NT = Lay::threads, RBK = Lay::RBK, PBK = kDeltaC * RBK;
    constexpr int NQ = DKP / 32;   // 8-column tiles of a warp's quarter of DK
    extern __shared__ __align__(128) unsigned char dsm[];
    const uint32_t sm0 = smem_addr(dsm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t2 = (lane & 3) * 2;
    const int gr = warp >> 2, w = warp & 3, b = (w + gr) & 3;   // group, quarter of DK, token block
    const int h = blockIdx.y, hk = h / (p.H / p.HK);
    const int dvw = (tile * GROUPS + gr) * 16;
    const bool won = dvw < (LOCAL && ident ? p.DK : p.DV);
    unsigned char *gb = dsm + Lay::oG + gr * Lay::group;
    const uint32_t sS = sm0 + Lay::oG + gr * Lay::group + Lay::gS, sX = sS + Lay::gX, sU = sS + Lay::gU;
    auto meet = [&] { asm volatile("bar.sync %0, 128;\n" ::"r"(1 + gr) : "memory"); };
    auto commit = [&] { asm volatile("cp.async.commit_group;\n" ::: "memory"); };
    __shared__ int ranked;
    for (long long z = blockIdx.z; z < units; z += gridDim.z) {
        // packed sequences are taken by length, the longest first
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

        // K or Q of chunk c
        auto load_rows = [&](int c, uint32_t dst0, const void *base, long long ts, const void *parts) {
            const int t0 = c * kDeltaC;
            for (int i = tid; i < NPI * kDeltaC * (DKP / 8); i += NT) {
                const int r = i / (DKP / 8), pc = i % (DKP / 8);   // r counts the parts' rows
                const char *src;
                bool on = true;
                if constexpr (NPI == 1) {
                    on = t0 + r < q.len && pc * 8 < p.DK;
                    src = static_cast<const char *>(base) +
                          (delta_token(p, q, on ? t0 + r : 0) * ts + (long long)hk * p.DK + (on ? pc * 8 : 0)) * 2;
                } else {
                    src = static_cast<const char *>(parts) + ((slot0 + c) * p.HK + hk) * (NPI * PBK) +
                          (long long)i * 16;
                }
                cp16(dst0 + (r / kDeltaC) * PBK + swz<RBK>(r % kDeltaC, pc), src, on);
            }
        };
        auto load_k = [&](int i) {   // and the decays; chunk i of the chain
            const int c = chunk(i);
            load_rows(c, sm0 + Lay::oK + (KBUF == 2 ? i & 1 : 0) * Lay::KB, p.k, p.ks, p.kp);
            if (tid < 48)
                cp16(sm0 + Lay::oVec + (i & 1) * 768 + tid * 16,
                     p.vec + ((slot0 + c) * p.H + h) * kDeltaVec + tid * 4, true);
        };
        auto load_vt = [&](int c) {
            const long long sh = (slot0 + c) * p.H + h;
            const int t0 = c * kDeltaC;
            constexpr int VPC = Lay::DVT * (int)sizeof(Tin) / 16, VPE = 16 / (int)sizeof(Tin);
            for (int i = tid; i < (LOCAL && ident ? 0 : kDeltaC * VPC); i += NT) {
                const int r = i / VPC, pc = i % VPC, d = tile * Lay::DVT + pc * VPE;
                const bool on = t0 + r < q.len && d < p.DV;
                const long long tok = delta_token(p, q, on ? t0 + r : 0);
                const Tin *src = MODE == kChainRev ? static_cast<const Tin *>(p.dout) + (tok * p.H + h) * p.DV
                                                   : static_cast<const Tin *>(p.v) + tok * p.vs + (long long)h * p.DV;
                cp16(sm0 + Lay::oV + r * Lay::VRB + pc * 16, src + (on ? d : 0), on);
            }
            for (int i = tid; i < NP * kTriBytes / 16; i += NT)
                cp16(sm0 + Lay::oT + i * 16, static_cast<const char *>(p.Tp) + sh * NP * kTriBytes + i * 16, true);
            if constexpr (MODE != kChainState)
                for (int i = tid; i < NPP * kTriBytes / 16; i += NT)
                    cp16(sm0 + Lay::oP + i * 16, static_cast<const char *>(p.Pp) + sh * NPP * kTriBytes + i * 16,
                         true);
        };
        // V or dO of the group's columns and token block blk, as an accumulator pair and as an A operand
        auto values = [&](int blk, float (&v)[2][4]) {
            if constexpr (sizeof(Tin) == 2) {
                uint32_t r[4];
                ldsm4t(sm0 + Lay::oV + (blk * 16 + (lane & 7) + (lane >> 4) * 8) * Lay::VRB + gr * 32 +
                           (lane >> 3 & 1) * 16,
                       r);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j >> 1][(j & 1) * 2] = half_bits_to_f32<Tin>(r[j] & 0xffffu);
                    v[j >> 1][(j & 1) * 2 + 1] = half_bits_to_f32<Tin>(r[j] >> 16);
                }
            } else {
                const float *vt = reinterpret_cast<const float *>(dsm + Lay::oV) + gr * 16;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[e][j] = vt[(blk * 16 + e * 8 + t2 + (j & 1)) * (Lay::DVT + 4) + g8 + (j >> 1) * 8];
            }
        };
        // N parts of a 16 x 16 accumulator pair into token block blk of a group's tile
        auto leave = [&](auto parts, int tile_, int blk, const float (&v)[2][4]) {
            constexpr int N = decltype(parts)::value;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t o[N];
                    split2<N>(v[e][hf * 2], v[e][hf * 2 + 1], o);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        *reinterpret_cast<uint32_t *>(gb + tile_ + m * Lay::XP + swz<128>(g8 + hf * 8, blk * 2 + e) +
                                                      t2 * 2) = o[m];
                }
        };
        // the A operand of token block blk of such a tile, of columns ks * 16.. of S
        auto take = [&](uint32_t tile_, int blk, auto &a) {
            constexpr int N = sizeof(a) / sizeof(a[0]);
#pragma unroll
            for (int m = 0; m < N; ++m)
                ldsm4(tile_ + m * Lay::XP + swz<128>(lane & 15, blk * 2 + (lane >> 4)), a[m]);
        };
        auto take_s = [&](int ks, auto &a) {
            constexpr int N = sizeof(a) / sizeof(a[0]);
#pragma unroll
            for (int m = 0; m < N; ++m)
                ldsm4(sS + m * Lay::SP + swz<RBK>(lane & 15, ks * 2 + (lane >> 4)), a[m]);
        };
        // a 16 x 16 result, transposed back and rounded, into the rows of a (tokens, H, DV) tensor
        auto emit = [&](const float (&v)[2][4], void *dst, int t0) {
            if constexpr (sizeof(Tin) == 2) {
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = v[j >> 1][(j & 1) * 2], y = v[j >> 1][(j & 1) * 2 + 1];
                    if constexpr (std::is_same_v<Tin, __half>) {
                        const __half2 hh = __floats2half2_rn(x, y);
                        r[j] = *reinterpret_cast<const uint32_t *>(&hh);
                    } else {
                        r[j] = pack_bf16(x, y);
                    }
                }
                const int eb = Lay::oE + warp * 512;
                stsm4t(sm0 + eb + ((lane & 7) + (lane >> 4) * 8) * 32 + (lane >> 3 & 1) * 16, r);
                __syncwarp();
                const int t = t0 + (lane >> 1);
                if (t < q.len)
                    *reinterpret_cast<uint4 *>(static_cast<Tin *>(dst) + (delta_token(p, q, t) * p.H + h) * p.DV +
                                               dvw + (lane & 1) * 8) =
                        *reinterpret_cast<const uint4 *>(dsm + eb + lane * 16);
                __syncwarp();
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = t0 + e * 8 + t2 + (j & 1);
                        if (t < q.len)
                            static_cast<Tin *>(dst)[(delta_token(p, q, t) * p.H + h) * p.DV + dvw + g8 +
                                                    (j >> 1) * 8] = v[e][j];
                    }
            }
        };
        // float pairs of a transposed scratch tile [DV][W], columns col..
        auto put = [&](float *dst, long long sh, int Wd, int col, const float (&v)[4]) {
            float *r = dst + (sh * p.DV + dvw + g8) * Wd + col + t2;
            *reinterpret_cast<float2 *>(r) = make_float2(v[0], v[1]);
            *reinterpret_cast<float2 *>(r + 8 * Wd) = make_float2(v[2], v[3]);
        };

        const int dk0 = w * (DKP / 4);
        float S[NQ][4];
        {
            const float *src = MODE == kChainRev ? p.dh_last : p.h0;
            const float *sin = (MODE == kChainRev ? p.dSin : p.Sin) + (su * p.DV + dvw + g8) * DKP;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int dk = dk0 + n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
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
        auto leave_s = [&] {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t o[NP];
                    split2<NP>(S[n][hf * 2], S[n][hf * 2 + 1], o);
#pragma unroll
                    for (int m = 0; m < NP; ++m)
                        *reinterpret_cast<uint32_t *>(gb + Lay::gS + m * Lay::SP +
                                                      swz<RBK>(g8 + hf * 8, w * NQ + n) + t2 * 2) = o[m];
                }
        };
        if (nc > 0) {
            load_k(0);
            leave_s();
        }
        commit();
        for (int i = 0; i < nc; ++i) {
            const int c = chunk(i), t0 = c * kDeltaC, nb = (min(q.len - t0, kDeltaC) + 15) / 16;
            const long long sh = (slot0 + c) * p.H + h;
            cp_wait();
            __syncthreads();   // K and the parts of S are here; everything of the last chunk is read
            load_vt(c);
            if constexpr (MODE != kChainState)
                load_rows(c, sm0 + Lay::oQ, p.q, p.qs, p.qp);
            commit();
            if (KBUF == 2 && i + 1 < nc)
                load_k(i + 1);
            commit();
            const uint32_t sK = sm0 + Lay::oK + (KBUF == 2 ? i & 1 : 0) * Lay::KB, sQ = sm0 + Lay::oQ;
            const float *eg = reinterpret_cast<const float *>(dsm + Lay::oVec + (i & 1) * 768);
            const float *el = eg + kDeltaC, *be = el + kDeltaC;
            const bool on = won && b < nb;   // a token block with tokens
            float R[2][4] = {}, U[2][4] = {};
            if (won) {
                if constexpr (MODE != kChainOut && !LOCAL) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        put(MODE == kChainRev ? p.dSx : p.Sx, sh, DKP, dk0 + n * 8, S[n]);
                }
            }
            if (on) {   // (K S)^T of the block
#pragma unroll
                for (int ks = 0; ks < DKP / 16; ++ks) {
                    uint32_t a[NP][4];
                    take_s(ks, a);
                    mma_rows<RBK, NP, NPI, NP>(R[0], R[1], a, sK, PBK, b * 16, ks * 2);
                }
            }
            asm volatile("cp.async.wait_group 1;\n" ::: "memory");
            __syncthreads();   // Q, T, P and V are here
            const int tb = b * 16 + t2;   // the lane's first token of the block
            if constexpr (MODE != kChainRev) {
                if (on) {
                    float v[2][4] = {};
                    if (!(LOCAL && ident))
                        values(b, v);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t = tb + e * 8 + (j & 1);
                            R[e][j] = be[t] * (v[e][j] - eg[t] * R[e][j]);   // X
                        }
                    leave(std::integral_constant<int, NP>(), Lay::gX, b, R);
                }
                meet();   // X is here
                if (on) {
                    // V'^T = X^T T^T
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j <= b) {
                            uint32_t a[NP][4];
                            take(sX, j, a);
                            mma_block_rows<NP, NP, NP>(U[0], U[1], a, sm0 + Lay::oT + tri_block(b, j));
                        }
                    if constexpr (MODE == kChainOut)
                        leave(std::integral_constant<int, NPP>(), Lay::gU, b, U);
                    else if constexpr (!LOCAL)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            put(p.Vx, sh, kDeltaC, b * 16 + e * 8, U[e]);
                }
                meet();   // X is read, V' is here
                if (on) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            U[e][j] *= el[tb + e * 8 + (j & 1)];
                    leave(std::integral_constant<int, NP>(), Lay::gX, b, U);
                    if constexpr (MODE == kChainOut) {
                        // O^T = scale e^c (Q S)^T + V'^T P^T
                        float O[2][4] = {};
#pragma unroll
                        for (int ks = 0; ks < DKP / 16; ++ks) {
                            uint32_t a[NPP][4];
                            take_s(ks, a);
                            mma_rows<RBK, NPP, NPI, NPP>(O[0], O[1], a, sQ, PBK, b * 16, ks * 2);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                O[e][j] *= p.scale * eg[tb + e * 8 + (j & 1)];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j <= b) {
                                uint32_t a[NPP][4];
                                take(sU, j, a);
                                mma_block_rows<NPP, NPP, NPP>(O[0], O[1], a, sm0 + Lay::oP + tri_block(b, j));
                            }
                        emit(O, p.o, t0 + b * 16);
                    }
                }
                meet();   // e^{c_last - c} V' is here, S is read
            } else {
                if (on) {
                    // dV'^T = dO^T P + e^{c_last - c} (K dS)^T
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[e][j] *= el[tb + e * 8 + (j & 1)];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k >= b && k < nb) {
                            float v[2][4];
                            values(k, v);
                            uint32_t a[NPI][4];
                            frag_a<NPI>(v[0], v[1], a);
                            mma_block_cols<NPI, NPP, NPP>(R[0], R[1], a, sm0 + Lay::oP + tri_block(k, b));
                        }
                    leave(std::integral_constant<int, NP>(), Lay::gX, b, R);
                }
                meet();   // dV' is here
                if (on) {
                    // dX^T = dV'^T T
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k >= b && k < nb) {
                            uint32_t a[NP][4];
                            take(sX, k, a);
                            mma_block_cols<NP, NP, NP>(U[0], U[1], a, sm0 + Lay::oT + tri_block(k, b));
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if constexpr (!LOCAL)
                            put(p.dXx, sh, kDeltaC, b * 16 + e * 8, U[e]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t = tb + e * 8 + (j & 1);
                            U[e][j] *= be[t];
                            R[e][j] = -eg[t] * U[e][j];   // dR
                        }
                    }
                    leave(std::integral_constant<int, NP>(), Lay::gU, b, R);
                    if constexpr (!LOCAL)
                        emit(U, p.dv, t0 + b * 16);
                }
                meet();   // dV' is read
                if (on) {
                    values(b, R);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            R[e][j] *= p.scale * eg[tb + e * 8 + (j & 1)];
                    leave(std::integral_constant<int, NP>(), Lay::gX, b, R);
                }
                meet();   // dR and scale e^c dO are here
            }
            if (won) {
                // S^T <- e^{c_last} S^T + (e^{c_last - c} V')^T K, or dR^T K + (scale e^c dO)^T Q
                const float elast = eg[kDeltaC - 1];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        S[n][j] *= elast;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < nb) {
                        uint32_t a[NP][4];
                        take(MODE == kChainRev ? sU : sX, k, a);
#pragma unroll
                        for (int nt = 0; nt < NQ; nt += 2)
                            mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sK, PBK, k * 16, w * NQ + nt);
                        if constexpr (MODE == kChainRev) {
                            take(sX, k, a);
#pragma unroll
                            for (int nt = 0; nt < NQ; nt += 2)
                                mma_cols<RBK, NP, NPI, NP>(S[nt], S[nt + 1], a, sQ, PBK, k * 16, w * NQ + nt);
                        }
                    }
                leave_s();
            }
            if (KBUF == 1 && i + 1 < nc) {
                __syncthreads();
                load_k(i + 1);
                commit();
            }
        }
        if constexpr (LOCAL) {
            if (won && ident) {
                uint32_t *m = static_cast<uint32_t *>(p.Ms);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    uint32_t x[3], y[3];
                    split2<3>(S[n][0], S[n][1], x);
                    split2<3>(S[n][2], S[n][3], y);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        uint32_t *r = m + (((su * 3 + k) * DKP + dvw + g8) * DKP + dk0 + n * 8 + t2) / 2;
                        r[0] = x[k];
                        r[8 * DKP / 2] = y[k];
                    }
                }
            } else if (won) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    put(MODE == kChainRev ? p.dNs : p.Ns, su, DKP, dk0 + n * 8, S[n]);
            }
        } else {
            float *dst = MODE == kChainRev ? p.dh0 : p.h_last;
            if (dst && won && (MODE == kChainRev ? c0 == 0 : c1 == nchunks)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int dk = dk0 + n * 8 + t2 + (j & 1), dv = dvw + g8 + (j >> 1) * 8;
                        if (dk < p.DK)
                            dst[(((long long)sn * p.H + h) * p.DK + dk) * p.DV + dv] = S[n][j];
                    }
            }
        }
        cp_wait();
        __syncthreads();
    }
}

template <typename Tin, int DKP, int GROUPS, int NP, int NPP, int KBUF>
__global__ void __launch_bounds__(GROUPS * 128, 1) delta_split_out_kernel(const DeltaParams p, long long units)
{
    delta_split<Tin, DKP, GROUPS, kChainOut, NP, NPP, KBUF, false>(p, blockIdx.x, false, units);
}
// both chains of the backward pass, the longer one first
template <typename Tin, int DKP, int GROUPS, int KBUF>
__global__ void __launch_bounds__(GROUPS * 128, 1) delta_split_both_kernel(const DeltaParams p, long long units)
{
    if (blockIdx.x & 1)
        delta_split<Tin, DKP, GROUPS, kChainState, 3, 3, KBUF, false>(p, blockIdx.x >> 1, false, units);
    else
        delta_split<Tin, DKP, GROUPS, kChainRev, 3, 3, KBUF, false>(p, blockIdx.x >> 1, false, units);
}
// first pass over the segments: tiles of DV forward, of DK for the transition, and of DV in reverse (REV)
template <typename Tin, int DKP, int GROUPS, int NP, int KBUF, bool REV>
__global__ void __launch_bounds__(GROUPS * 128, 1)
    delta_split_local_kernel(const DeltaParams p, int dvt, int dkt, long long units)
{
    const int x = blockIdx.x;
    if (x < dvt + dkt)
        delta_split<Tin, DKP, GROUPS, kChainState, NP, 3, KBUF, true>(p, x < dvt ? x : x - dvt, x >= dvt, units,
                                                                      REV && x >= dvt);
    else if constexpr (REV)
        delta_split<Tin, DKP, GROUPS, kChainRev, NP, 3, KBUF, true>(p, x - dvt - dkt, false, units);
}

}  // namespace ss2d
