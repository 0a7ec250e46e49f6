// ss2d_delta_grad.cuh -- the gradients of a chunk's tokens, once the states
// before and their gradients after every chunk are known.
//
// With S before and dS after the chunk, dX and V' from the chains
// (ss2d_delta_chain.cuh), per head:
//     dP = dO V'^T (i >= j),   dA = -dX V'^T (i > j)
//     GP = scale D dP,         GA = beta D dA,     E = dP P + dA A
//     dq = scale e^c (dO S^T) + GP K
//     dk = dR S^T + e^{c_last - c} (V' dS^T) + GP^T Q + GA K + GA^T K
//     dbeta = dX.Y + sum_j D (k.k) dA
//     dc = row sums of E - column sums of E + q.(scale e^c dO S^T) + dR.(K S) - kl,
//          and on the last token sum kl + e^{c_last} S.dS,    kl = e^{c_last - c} V'.(K dS)
//     dg = sums of dc from the chunk's end
// (dv = beta dX is written by the reverse chain.)  A CTA of 8 warps has one
// (slot, key head) and goes through its value heads in order, so that the
// gradients of shared keys and queries are sums in a fixed order: warp w
// holds rows 16 (w % 4) .. + 15 and half w / 4 of the columns of dq, dk (over DK)
// and of dP, dA (over tokens).  DV is gone through in tiles of 32 columns,
// split into bf16 parts as they are staged.  What reaches a float32 output (dq's
// first term and E, through dg) keeps three parts, dk and the second term of dq
// two when they are stored in 16 bits.
#pragma once

#include "ss2d_delta_chain.cuh"

namespace ss2d {

constexpr int kGradThreads = 256;
constexpr int kGradDV = 32;      // DV columns per staged tile
constexpr int kGradORow = kGradDV * 2 + 16;   // bytes of a staged dO row

template <typename Tin, int DKP>
struct GradLayout {
    static constexpr int NPI = DeltaParts<Tin>::n, NP = 3, NPG = sizeof(Tin) == 2 ? 2 : 3;
    static constexpr int RBK = DKP * 2, PBK = kDeltaC * RBK;
    static constexpr int SB = kGradDV * RBK;         // one part of S^T or dS^T
    static constexpr int XB = kGradDV * 128;         // one part of dX, V'
    static constexpr int GB = kDeltaC * 128;         // one part of GP, GA
    static constexpr int oK = 0, oQ = NPI * PBK, oS = 2 * NPI * PBK;
    static constexpr int sS = (NP + NPG) * SB > 2 * NPG * GB ? (NP + NPG) * SB : 2 * NPG * GB;   // GP, GA in its place
    static constexpr int oO = oS + sS;
    static constexpr int oX = oO + NPI * kDeltaC * kGradORow;
    static constexpr int oV = oX + NP * XB;
    static constexpr int oXs = oV + NP * XB;
    static constexpr int oVs = oXs + NPG * XB;
    static constexpr int bytes = oVs + NPG * XB;
};

// 8 floats as the parts of a swizzled row piece
template <int N, int RB>
__device__ __forceinline__ void put_parts(unsigned char *tile, int part, int r, int pc, const float (&v)[8])
{
    uint32_t w[4][N];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        split2<N>(v[2 * j], v[2 * j + 1], w[j]);
#pragma unroll
    for (int n = 0; n < N; ++n)
        *reinterpret_cast<uint4 *>(tile + n * part + swz<RB>(r, pc)) = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
}
__device__ __forceinline__ void load8(const float *src, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
}
template <typename Tin, int DKP>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const DeltaParams p)
{
    using Lay = GradLayout<Tin, DKP>;
    constexpr int NPI = Lay::NPI, NP = Lay::NP, NPG = Lay::NPG, RBK = Lay::RBK, PBK = Lay::PBK;
    constexpr int NH = DKP / 16;   // 8-column tiles of a warp's half of DK
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ float ch[kDeltaC], cl[kDeltaC], be[kDeltaC];
    __shared__ float red[8][2][kDeltaC];                     // token sums over the warps' rows of a tile
    __shared__ float rowE[2][kDeltaC], rowB[2][kDeltaC], rowQ[2][kDeltaC], colE[4][kDeltaC], rsd[8];
    int s, c;
    DeltaSeq q;
    if (!delta_slot(p, blockIdx.x, s, q, c))
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t2 = (lane & 3) * 2;
    const int wr = warp & 3, wc = warp >> 2;
    const int hk = blockIdx.y, G = p.H / p.HK, t0 = c * kDeltaC;
    const uint32_t sa = smem_addr(dsm);
    delta_stage_parts<Tin, DKP, NPI>(p, p.k, p.ks, hk, q, t0, dsm + Lay::oK, kGradThreads);
    delta_stage_parts<Tin, DKP, NPI>(p, p.q, p.qs, hk, q, t0, dsm + Lay::oQ, kGradThreads);
    __syncthreads();
    float kk[4][4], qk[4][4], dqt[NH][4], dk[NH][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            kk[n][j] = qk[n][j] = 0.f;
#pragma unroll
        for (int n = 0; n < NH; ++n)
            dqt[n][j] = dk[n][j] = 0.f;
    }
    delta_rows_product<DKP, NPI, 4>(sa + Lay::oK, sa + Lay::oK, wr * 16, wc * 32, kk);
    delta_rows_product<DKP, NPI, 4>(sa + Lay::oQ, sa + Lay::oK, wr * 16, wc * 32, qk);
    const int i0 = wr * 16 + g8;   // the lane's rows: i0, i0 + 8

    for (int hi = 0; hi < G; ++hi) {
        const int h = hk * G + hi;
        const long long sh = (long long)blockIdx.x * p.H + h;
        const float *vec = p.vec + sh * 3 * kDeltaC;
        __syncthreads();
        if (warp == 0)
            delta_decays(p, q, t0, h, ch, cl, be);
        float dq[NH][4], dP[4][4], dA[4][4], bd[8], rd[8], sd = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                dP[n][j] = dA[n][j] = 0.f;
#pragma unroll
            for (int n = 0; n < NH; ++n)
                dq[n][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            bd[j] = rd[j] = 0.f;
        // a thread's piece of a token tile: 8 tokens from tk of row tr
        const int tr = tid >> 3, tk = (tid & 7) * 8;
        float fx[8], fv[8];   // -beta e^c and e^{c_last - c} of the tokens
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            fx[j] = -vec[2 * kDeltaC + tk + j] * vec[tk + j];
            fv[j] = vec[kDeltaC + tk + j];
        }
        for (int d0 = 0; d0 < p.DV; d0 += kGradDV) {
            __syncthreads();
            // S^T, dS^T
            for (int i = tid; i < kGradDV * (DKP / 8); i += kGradThreads) {
                const int r = i / (DKP / 8), pc = i % (DKP / 8);
                float a[8], b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    a[j] = b[j] = 0.f;
                if (d0 + r < p.DV) {
                    const long long o = (sh * p.DV + d0 + r) * DKP + pc * 8;
                    load8(p.Sx + o, a);
                    load8(p.dSx + o, b);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sd = fmaf(a[j], b[j], sd);
                put_parts<NP, RBK>(dsm + Lay::oS, Lay::SB, r, pc, a);
                put_parts<NPG, RBK>(dsm + Lay::oS + NP * Lay::SB, Lay::SB, r, pc, b);
            }
            {   // dX, V' and their scaled forms; dX.Y and dX.(e^c K S) with e^c K S = V - Y
                float x[8], v[8], y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = v[j] = 0.f;
                if (d0 + tr < p.DV) {
                    const long long o = (sh * p.DV + d0 + tr) * kDeltaC + tk;
                    load8(p.dXx + o, x);
                    load8(p.Vx + o, v);
                    load8(p.Yx + o, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = t0 + tk + j;
                        const float vi = t < q.len ? to_f32(static_cast<const Tin *>(p.v)[delta_token(p, q, t) * p.vs +
                                                                                          (long long)h * p.DV + d0 + tr])
                                                   : 0.f;
                        bd[j] = fmaf(x[j], y[j], bd[j]);
                        rd[j] = fmaf(x[j], vi - y[j], rd[j]);
                    }
                }
                put_parts<NP, 128>(dsm + Lay::oX, Lay::XB, tr, tid & 7, x);
                put_parts<NP, 128>(dsm + Lay::oV, Lay::XB, tr, tid & 7, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] *= fx[j];
                    v[j] *= fv[j];
                }
                put_parts<NPG, 128>(dsm + Lay::oXs, Lay::XB, tr, tid & 7, x);
                put_parts<NPG, 128>(dsm + Lay::oVs, Lay::XB, tr, tid & 7, v);
            }
            {   // dO: rows of 32 columns
                const int r = tid >> 2, pc = tid & 3, t = t0 + r, d = d0 + pc * 8;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = 0.f;
                if (t < q.len && d < p.DV) {
                    const Tin *row = static_cast<const Tin *>(p.dout) + (delta_token(p, q, t) * p.H + h) * p.DV + d;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = to_f32(row[j]);
                }
                uint32_t w[4][NPI];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    split2<NPI>(v[2 * j], v[2 * j + 1], w[j]);
#pragma unroll
                for (int n = 0; n < NPI; ++n)
                    *reinterpret_cast<uint4 *>(dsm + Lay::oO + (n * kDeltaC + r) * kGradORow + pc * 16) =
                        make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
            }
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < kGradDV / 16; ++ks) {
                uint32_t ao[NPI][4], ax[NP][4];
#pragma unroll
                for (int n = 0; n < NPI; ++n)
                    ldsm4(sa + Lay::oO + (n * kDeltaC + wr * 16 + (lane & 15)) * kGradORow +
                              (ks * 2 + (lane >> 4)) * 16,
                          ao[n]);
#pragma unroll
                for (int nt = 0; nt < NH; nt += 2)
                    mma_cols<RBK, NPI, NP, NP>(dq[nt], dq[nt + 1], ao, sa + Lay::oS, Lay::SB, ks * 16, wc * NH + nt);
                frag_t<NP>(sa + Lay::oX, Lay::XB, ks * 16, wr * 16, ax);
#pragma unroll
                for (int nt = 0; nt < 4; nt += 2) {
                    if (wc * 2 + nt / 2 <= wr) {   // blocks above the diagonal are not needed
                        mma_cols<128, NPI, NP, NP>(dP[nt], dP[nt + 1], ao, sa + Lay::oV, Lay::XB, ks * 16,
                                                   wc * 4 + nt);
                        mma_cols<128, NP, NP, NP>(dA[nt], dA[nt + 1], ax, sa + Lay::oV, Lay::XB, ks * 16,
                                                  wc * 4 + nt);
                    }
                }
                uint32_t as[NPG][4];
                frag_t<NPG>(sa + Lay::oXs, Lay::XB, ks * 16, wr * 16, as);
#pragma unroll
                for (int nt = 0; nt < NH; nt += 2)
                    mma_cols<RBK, NPG, NPG, NPG>(dk[nt], dk[nt + 1], as, sa + Lay::oS, Lay::SB, ks * 16, wc * NH + nt);
                frag_t<NPG>(sa + Lay::oVs, Lay::XB, ks * 16, wr * 16, as);
#pragma unroll
                for (int nt = 0; nt < NH; nt += 2)
                    mma_cols<RBK, NPG, NPG, NPG>(dk[nt], dk[nt + 1], as, sa + Lay::oS + NP * Lay::SB, Lay::SB, ks * 16,
                                                 wc * NH + nt);
            }
        }
        // sums of the staged pieces: over a warp's four rows, then the warps
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            for (int m = 8; m < 32; m <<= 1) {
                bd[j] += __shfl_xor_sync(0xffffffffu, bd[j], m);
                rd[j] += __shfl_xor_sync(0xffffffffu, rd[j], m);
            }
            if (lane < 8) {
                red[warp][0][tk + j] = bd[j];
                red[warp][1][tk + j] = rd[j];
            }
        }
        for (int m = 1; m < 32; m <<= 1)
            sd += __shfl_xor_sync(0xffffffffu, sd, m);
        if (lane == 0)
            rsd[warp] = sd;
        // dq's first term and its product with q
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const float f = p.scale * vec[i0 + hf * 8];
            float dot = 0.f;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                float q0 = 0.f, q1 = 0.f;
#pragma unroll
                for (int n = NPI - 1; n >= 0; --n) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(
                        dsm + Lay::oQ + n * PBK + swz<RBK>(i0 + hf * 8, wc * NH + nt) + t2 * 2);
                    q0 += __uint_as_float(w << 16);
                    q1 += __uint_as_float(w & 0xffff0000u);
                }
                const float a = f * dq[nt][hf * 2], b = f * dq[nt][hf * 2 + 1];
                dot = fmaf(a, q0, fmaf(b, q1, dot));
                dqt[nt][hf * 2] += a;
                dqt[nt][hf * 2 + 1] += b;
            }
            dot += __shfl_xor_sync(0xffffffffu, dot, 1);
            dot += __shfl_xor_sync(0xffffffffu, dot, 2);
            if ((lane & 3) == 0)
                rowQ[wc][i0 + hf * 8] = dot;
        }
        __syncthreads();   // every warp is done with S^T: GP and GA take its place
        unsigned char *gp = dsm + Lay::oS, *ga = gp + NPG * Lay::GB;
        float ce[4][2];
        float re[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int j0 = wc * 32 + n * 8 + t2;
            ce[n][0] = ce[n][1] = 0.f;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = i0 + hf * 8;
                float vp[2], va[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + e, x = hf * 2 + e;
                    vp[e] = va[e] = 0.f;
                    if (j <= i) {
                        const float D = expf((ch[i] - ch[j]) + (cl[i] - cl[j]));
                        vp[e] = p.scale * D * dP[n][x];
                        float E = vp[e] * qk[n][x];
                        if (j < i) {
                            const float Dk = D * kk[n][x], da = -dA[n][x];
                            va[e] = be[i] * D * da;
                            E = fmaf(be[i] * Dk, da, E);
                            rb[hf] = fmaf(Dk, da, rb[hf]);
                        }
                        re[hf] += E;
                        ce[n][e] += E;
                    }
                }
                uint32_t w[NPG];
                const uint32_t o = swz<128>(i, wc * 4 + n) + t2 * 2;
                split2<NPG>(vp[0], vp[1], w);
#pragma unroll
                for (int m = 0; m < NPG; ++m)
                    *reinterpret_cast<uint32_t *>(gp + m * Lay::GB + o) = w[m];
                split2<NPG>(va[0], va[1], w);
#pragma unroll
                for (int m = 0; m < NPG; ++m)
                    *reinterpret_cast<uint32_t *>(ga + m * Lay::GB + o) = w[m];
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            for (int m = 1; m < 4; m <<= 1) {
                re[hf] += __shfl_xor_sync(0xffffffffu, re[hf], m);
                rb[hf] += __shfl_xor_sync(0xffffffffu, rb[hf], m);
            }
            if ((lane & 3) == 0) {
                rowE[wc][i0 + hf * 8] = re[hf];
                rowB[wc][i0 + hf * 8] = rb[hf];
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                for (int m = 4; m < 32; m <<= 1)
                    ce[n][e] += __shfl_xor_sync(0xffffffffu, ce[n][e], m);
                if (g8 == 0)
                    colE[wr][wc * 32 + n * 8 + t2 + e] = ce[n][e];
            }
        __syncthreads();
        if (warp == 0) {
            // dc, dbeta; then sums of dc from the end: lane l holds tokens 2l, 2l + 1
            float dc[2], kls = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float b = 0.f, r = 0.f, kl = 0.f;
                for (int w = 0; w < 8; ++w) {
                    b += red[w][0][i];
                    r += red[w][1][i];
                }
                for (int w = 0; w < p.DV / 16; ++w)
                    kl += p.klx[(sh * (p.DV / 16) + w) * kDeltaC + i];
                kls += kl;
                const float E = (rowE[0][i] + rowE[1][i]) - ((colE[0][i] + colE[1][i]) + (colE[2][i] + colE[3][i]));
                dc[e] = ((E + (rowQ[0][i] + rowQ[1][i])) - be[i] * r) - kl;
                if (t0 + i < q.len)
                    p.dbeta[delta_token(p, q, t0 + i) * p.H + h] = b + (rowB[0][i] + rowB[1][i]);
            }
            for (int m = 1; m < 32; m <<= 1)
                kls += __shfl_xor_sync(0xffffffffu, kls, m);
            if (lane == 31) {
                float t = 0.f;
                for (int w = 0; w < 8; ++w)
                    t += rsd[w];
                dc[1] += kls + vec[kDeltaC - 1] * t;
            }
            float sum = dc[0] + dc[1];
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_down_sync(0xffffffffu, sum, o);
                if (lane + o < 32)
                    sum += u;
            }
            float after = __shfl_down_sync(0xffffffffu, sum, 1);
            after = (lane < 31 ? after : 0.f) + dc[1];
            if (t0 + 2 * lane < q.len)
                p.dg[delta_token(p, q, t0 + 2 * lane) * p.H + h] = after + dc[0];
            if (t0 + 2 * lane + 1 < q.len)
                p.dg[delta_token(p, q, t0 + 2 * lane + 1) * p.H + h] = after;
        }
        // GP K into dq; GP^T Q, GA K, GA^T K into dk
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t a[NPG][4], b[NPG][4];
            if (ks <= wr) {
                frag_n<NPG>(smem_addr(gp), Lay::GB, wr * 16, ks * 16, a);
                frag_n<NPG>(smem_addr(ga), Lay::GB, wr * 16, ks * 16, b);
#pragma unroll
                for (int nt = 0; nt < NH; nt += 2) {
                    mma_cols<RBK, NPG, NPI, NPG>(dqt[nt], dqt[nt + 1], a, sa + Lay::oK, PBK, ks * 16, wc * NH + nt);
                    mma_cols<RBK, NPG, NPI, NPG>(dk[nt], dk[nt + 1], b, sa + Lay::oK, PBK, ks * 16, wc * NH + nt);
                }
            }
            if (ks >= wr) {
                frag_t<NPG>(smem_addr(gp), Lay::GB, ks * 16, wr * 16, a);
                frag_t<NPG>(smem_addr(ga), Lay::GB, ks * 16, wr * 16, b);
#pragma unroll
                for (int nt = 0; nt < NH; nt += 2) {
                    mma_cols<RBK, NPG, NPI, NPG>(dk[nt], dk[nt + 1], a, sa + Lay::oQ, PBK, ks * 16, wc * NH + nt);
                    mma_cols<RBK, NPG, NPI, NPG>(dk[nt], dk[nt + 1], b, sa + Lay::oK, PBK, ks * 16, wc * NH + nt);
                }
            }
        }
    }
    auto store = [&](void *dst, const float (&v)[NH][4]) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int t = t0 + i0 + hf * 8;
            if (t >= q.len)
                continue;
            Tin *row = static_cast<Tin *>(dst) + (delta_token(p, q, t) * p.HK + hk) * p.DK;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const int d = (wc * NH + nt) * 8 + t2;
                if (d >= p.DK)
                    continue;
                const float a = v[nt][hf * 2], b = v[nt][hf * 2 + 1];
                if constexpr (std::is_same_v<Tin, float>) {
                    *reinterpret_cast<float2 *>(row + d) = make_float2(a, b);
                } else if constexpr (std::is_same_v<Tin, __half>) {
                    const __half2 hh = __floats2half2_rn(a, b);
                    *reinterpret_cast<uint32_t *>(row + d) = *reinterpret_cast<const uint32_t *>(&hh);
                } else {
                    *reinterpret_cast<uint32_t *>(row + d) = pack_bf16(a, b);
                }
            }
        }
    };
    store(p.dq, dqt);
    store(p.dk, dk);
}

}  // namespace ss2d
