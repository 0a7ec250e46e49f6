// ss2d_delta_grad.cuh -- the gradients of a chunk's tokens, once the states
// before and their gradients after every chunk are known.
//
// With S before and dS after the chunk, dX and V' from the chains
// (ss2d_delta_chain.cuh), per head:
//     dP = dO V'^T (i >= j),   dA = -dX V'^T (i > j)
//     GP = scale D dP,         GA = beta D dA,     E = dP P + dA A
//     dq = scale e^c (dO S^T) + GP K
//     dk = dR S^T + e^{c_last - c} (V' dS^T) + GP^T Q + GA K + GA^T K,   dR = -beta e^c dX
//     rd = e^c k.(dX S^T),     dbeta = dX.V - rd + sum_j D (k.k) dA
//     dc = row sums of E - column sums of E + q.(scale e^c dO S^T) - beta rd - kl,
//          and on the last token sum kl + e^{c_last} S.dS,    kl = k.(e^{c_last - c} V' dS^T)
//     dg = sums of dc from the chunk's end
// (dv = beta dX is written by the reverse chain.)  A CTA of
// 8 warps has one (slot, key head) and goes through its value heads in order, so that the
// gradients of shared keys and queries are sums in a fixed order: warp w
// holds rows 16 (w % 4) .. + 15 and half w / 4 of the columns of dq, dk (over DK)
// and of dP, dA (over tokens).  DV is gone through in tiles of 32 columns:
// the tiles of S, dS, dX, V', dO and V are copied asynchronously while the tile
// before is multiplied, and split into bf16 parts when they are here (dX.V is summed
// from the copies).  What reaches a
// float32 output through dg and dbeta keeps three parts; the products with GP and
// GA two when dq and dk are stored in 16 bits.  Rows of tokens behind the end take no part.
//
// Heads of up to 64 in bfloat16 run two CTAs per SM (128 registers): with one, the kernel
// stood at 16 % of the tensor pipe, waiting on its staging (808 us for 6144
// chunks of 64 x 64 heads).  With two it took 412; of a CTA's 37,000 clocks the products
// had 16,000, the sums of E 6,500, most of them in branches, and staging 4,500: a tile of
// S^T or V' read once for two products, selects in place of the branches and dc
// and dbeta by two warps made it 364 (31,000 clocks; the tensor pipe at 37 %, issue at 43 %).
#pragma once

#include "ss2d_delta_chain.cuh"

namespace ss2d {

constexpr int kGradThreads = 256;

template <typename Tin, int DKP>
struct GradLayout {
    static constexpr int NPI = DeltaParts<Tin>::n, NPG = sizeof(Tin) == 2 ? 2 : 3;
    static constexpr int DVB = sizeof(Tin) == 4 && DKP == 128 ? 16 : 32;   // DV columns per staged tile
    static constexpr int ORow = DVB * 2 + 16;        // bytes of a staged row of dO
    static constexpr int RBK = DKP * 2, PBK = kDeltaC * RBK;
    static constexpr int SB = DVB * RBK;             // one part of S^T or dS^T
    static constexpr int XB = DVB * 128;             // one part of dX, V'
    static constexpr int oK = 0, oQ = NPI * PBK, oS = 2 * NPI * PBK;
    static constexpr int sG = 2 * NPG * kTriBytes;   // GP and GA, in the place of S^T and dS^T
    static constexpr int sS = 6 * SB > sG ? 6 * SB : sG;
    static constexpr int oO = oS + sS;
    static constexpr int oX = oO + NPI * kDeltaC * ORow;
    static constexpr int oV = oX + 3 * XB;
    static constexpr int oR = oV + 3 * XB;           // the next tile as it is: S^T, dS^T, dX, V', dO, V
    static constexpr int rS = DVB * DKP * 4, rX = DVB * kDeltaC * 4, rO = DVB * kDeltaC * (int)sizeof(Tin);
    static constexpr int PO = DVB * (int)sizeof(Tin) / 16;   // 16-byte pieces of a raw row of dO or V
    static constexpr int bytes = oR + 2 * rS + 2 * rX + 2 * rO;
    static constexpr int oE = oX;                    // sums of E, in the place of dX
    // place of piece pc of token t in a raw tile of dO or V: eight tokens' same pieces in eight bank groups
    static __device__ __forceinline__ int piece(int t, int pc) { return t * PO + (pc ^ (t / (8 / PO) & (PO - 1))); }
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
// 8 input values of a raw tile
template <typename Tin>
struct Piece8 {
    static constexpr int n = sizeof(Tin) / 2;
    uint4 u[n];
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (n == 2) {
                    v[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    v[2 * j] = half_bits_to_f32<Tin>(w[j] & 0xffffu);
                    v[2 * j + 1] = half_bits_to_f32<Tin>(w[j] >> 16);
                }
            }
        }
    }
};
// the parts of such a piece, `part` bytes apart
template <typename Tin, int NPI>
__device__ __forceinline__ void put_piece(unsigned char *dst, int part, const Piece8<Tin> &p)
{
    if constexpr (NPI == 1) {
        *reinterpret_cast<uint4 *>(dst) = p.u[0];
    } else {
        float v[8];
        p.get(v);
        uint32_t w[4][NPI];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            split2<NPI>(v[2 * j], v[2 * j + 1], w[j]);
#pragma unroll
        for (int n = 0; n < NPI; ++n)
            *reinterpret_cast<uint4 *>(dst + n * part) = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
    }
}

// SHARED: several value heads share the key head
template <typename Tin, int DKP, bool SHARED>
__global__ void __launch_bounds__(kGradThreads, (GradLayout<Tin, DKP>::bytes <= 109 * 1024 ? 2 : 1))
    delta_grad_kernel(const DeltaParams p)
{
    using Lay = GradLayout<Tin, DKP>;
    constexpr int NPI = Lay::NPI, NPG = Lay::NPG, RBK = Lay::RBK, PBK = Lay::PBK, DVB = Lay::DVB;
    constexpr int NH = DKP / 16;   // 8-column tiles of a warp's half of DK
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ __align__(16) float vec[kDeltaVec];   // e^c, e^{c_last - c}, beta, c and what it lacks
    const float *be = vec + 2 * kDeltaC, *ch = vec + 3 * kDeltaC, *cl = vec + 4 * kDeltaC;
    __shared__ float xv[4][kDeltaC], rowR[2][kDeltaC], rsd[8];
    __shared__ float rowQ[2][kDeltaC], rowK[2][kDeltaC];
    float(*rowE)[kDeltaC] = reinterpret_cast<float(*)[kDeltaC]>(dsm + Lay::oE), (*rowB)[kDeltaC] = rowE + 2,
    (*colE)[kDeltaC] = rowE + 4;
    int s, c;
    DeltaSeq q;
    if (!delta_slot(p, blockIdx.x, s, q, c))
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t2 = (lane & 3) * 2;
    const int wr = warp & 3, wc = warp >> 2;
    const int hk = blockIdx.y, G = p.H / p.HK, t0 = c * kDeltaC;
    const int nb = (min(q.len - t0, kDeltaC) + 15) / 16;   // blocks of 16 tokens that hold tokens
    const bool act = wr < nb;
    const uint32_t sa = smem_addr(dsm);
    const int tiles = (p.DV + DVB - 1) / DVB;
    // copies the raw tile n (head by head) of the group, rows past DV zero: S^T and dS^T; dX, V', dO and V
    auto raw_states = [&](int n) {
        const long long sh = (long long)blockIdx.x * p.H + hk * G + n / tiles;
        const int d0 = n % tiles * DVB;
        constexpr int PS = DKP / 4;   // 16-byte pieces of a row
#pragma unroll 4
        for (int i = tid; i < DVB * PS; i += kGradThreads) {
            const bool on = d0 + i / PS < p.DV;
            const long long o = (sh * p.DV + d0) * DKP + (on ? i * 4 : 0);
            cp16(sa + Lay::oR + i * 16, p.Sx + o, on);
            cp16(sa + Lay::oR + Lay::rS + i * 16, p.dSx + o, on);
        }
    };
    auto raw_tokens = [&](int n) {
        const long long sh = (long long)blockIdx.x * p.H + hk * G + n / tiles;
        const int d0 = n % tiles * DVB;
        constexpr int PX = kDeltaC / 4;
#pragma unroll 2
        for (int i = tid; i < DVB * PX; i += kGradThreads) {
            const bool on = d0 + i / PX < p.DV;
            const long long o = (sh * p.DV + d0) * kDeltaC + (on ? i * 4 : 0);
            cp16(sa + Lay::oR + 2 * Lay::rS + i * 16, p.dXx + o, on);
            cp16(sa + Lay::oR + 2 * Lay::rS + Lay::rX + i * 16, p.Vx + o, on);
        }
        const int h = hk * G + n / tiles;
        for (int i = tid; i < kDeltaC * Lay::PO; i += kGradThreads) {
            const int t = i / Lay::PO, pc = i % Lay::PO, d = d0 + pc * (16 / (int)sizeof(Tin));
            const bool on = t0 + t < q.len && d < p.DV;
            const long long tok = delta_token(p, q, on ? t0 + t : 0);
            const uint32_t at = sa + Lay::oR + 2 * Lay::rS + 2 * Lay::rX + Lay::piece(t, pc) * 16;
            cp16(at, static_cast<const Tin *>(p.dout) + (tok * p.H + h) * p.DV + (on ? d : 0), on);
            cp16(at + Lay::rO, static_cast<const Tin *>(p.v) + tok * p.vs + (long long)h * p.DV + (on ? d : 0), on);
        }
    };
    delta_stage_parts<Tin, DKP, NPI, kGradThreads>(p, p.k, p.ks, hk, q, t0, dsm + Lay::oK);
    delta_stage_parts<Tin, DKP, NPI, kGradThreads>(p, p.q, p.qs, hk, q, t0, dsm + Lay::oQ);
    raw_states(0);
    raw_tokens(0);
    float dqt[SHARED ? NH : 1][4], dkt[SHARED ? NH : 1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int n = 0; n < (SHARED ? NH : 1); ++n)
            dqt[n][j] = dkt[n][j] = 0.f;
    }
    const int ft = tid & 63, fp = tid >> 6;   // a thread's piece of dO and V: 8 columns from fp * 8 of token ft
    const int i0 = wr * 16 + g8;   // the lane's rows: i0, i0 + 8
    // the lane's two values of row i, tile nt of its half, of the staged q or k
    auto pair = [&](int tile, int i, int nt) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int n = NPI - 1; n >= 0; --n) {
            const uint32_t w =
                *reinterpret_cast<const uint32_t *>(dsm + tile + n * PBK + swz<RBK>(i, wc * NH + nt) + t2 * 2);
            v.x += __uint_as_float(w << 16);
            v.y += __uint_as_float(w & 0xffff0000u);
        }
        return v;
    };
    float dq[NH][4], dk[NH][4];
    for (int hi = 0; hi < G; ++hi) {
        const int h = hk * G + hi;
        const long long sh = (long long)blockIdx.x * p.H + h;
        __syncthreads();
        if (tid < kDeltaVec / 4)
            cp16(smem_addr(vec) + tid * 16, p.vec + sh * kDeltaVec + tid * 4, true);
        float dk2[NH][4], dP[4][4], dA[4][4], xd = 0.f, sd = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                dP[n][j] = dA[n][j] = 0.f;
#pragma unroll
            for (int n = 0; n < NH; ++n)
                dq[n][j] = dk[n][j] = dk2[n][j] = 0.f;
        }
        const int tr = tid >> 3, tk = (tid & 7) * 8;   // a thread's piece of a token tile: 8 tokens from tk of row tr
        for (int ti = 0; ti < tiles; ++ti) {
            cp_wait();
            __syncthreads();   // the raw tile is here, the last tile's parts are read
            const float *rs = reinterpret_cast<const float *>(dsm + Lay::oR);
            if (fp < DVB / 8) {
                const uint4 *ro = reinterpret_cast<const uint4 *>(rs + Lay::rS / 2 + Lay::rX / 2);
                Piece8<Tin> u;
#pragma unroll
                for (int i = 0; i < u.n; ++i)
                    u.u[i] = ro[Lay::piece(ft, fp * u.n + i)];
                put_piece<Tin, NPI>(dsm + Lay::oO + ft * Lay::ORow + fp * 16, kDeltaC * Lay::ORow, u);
#pragma unroll
                for (int i = 0; i < u.n; ++i)
                    u.u[i] = ro[Lay::rO / 16 + Lay::piece(ft, fp * u.n + i)];
                float x[8];
                u.get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    xd = fmaf(rs[Lay::rS / 2 + (fp * 8 + j) * kDeltaC + ft], x[j], xd);
            }
            for (int i = tid; i < DVB * (DKP / 8); i += kGradThreads) {
                const int r = i / (DKP / 8), pc = i % (DKP / 8);
                float a[8], b[8];
                load8(rs + i * 8, a);
                load8(rs + Lay::rS / 4 + i * 8, b);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sd = fmaf(a[j], b[j], sd);
                put_parts<3, RBK>(dsm + Lay::oS, Lay::SB, r, pc, a);
                put_parts<3, RBK>(dsm + Lay::oS + 3 * Lay::SB, Lay::SB, r, pc, b);
            }
            if (tr < DVB) {
                float x[8];
                load8(rs + Lay::rS / 2 + tr * kDeltaC + tk, x);
                put_parts<3, 128>(dsm + Lay::oX, Lay::XB, tr, tid & 7, x);
                load8(rs + Lay::rS / 2 + Lay::rX / 4 + tr * kDeltaC + tk, x);
                put_parts<3, 128>(dsm + Lay::oV, Lay::XB, tr, tid & 7, x);
            }
            __syncthreads();   // the parts are here, the raw tile is free
            const bool more = hi * tiles + ti + 1 < G * tiles;
            if (more)
                raw_states(hi * tiles + ti + 1);
#pragma unroll
            for (int ks = 0; ks < DVB / 16; ++ks) {
                if (act) {
                    {
                        // a tile of S^T serves dq and dk, one of V' dP and dA
                        uint32_t ao[NPI][4], ax[3][4], b[3][4];
#pragma unroll
                        for (int n = 0; n < NPI; ++n)
                            ldsm4(sa + Lay::oO + (n * kDeltaC + wr * 16 + (lane & 15)) * Lay::ORow +
                                      (ks * 2 + (lane >> 4)) * 16,
                                  ao[n]);
                        frag_t<3>(sa + Lay::oX, Lay::XB, ks * 16, wr * 16, ax);
#pragma unroll
                        for (int nt = 0; nt < NH; nt += 2) {
                            frag_cols<RBK, 3>(sa + Lay::oS, Lay::SB, ks * 16, wc * NH + nt, b);
                            mma_parts<NPI, 3, 3>(dq[nt], dq[nt + 1], ao, b);
                            mma_parts<3, 3, 3>(dk[nt], dk[nt + 1], ax, b);
                        }
#pragma unroll
                        for (int nt = 0; nt < 4; nt += 2)
                            if (wc * 2 + nt / 2 <= wr) {   // blocks above the diagonal are not needed
                                frag_cols<128, 3>(sa + Lay::oV, Lay::XB, ks * 16, wc * 4 + nt, b);
                                mma_parts<NPI, 3, 3>(dP[nt], dP[nt + 1], ao, b);
                                mma_parts<3, 3, 3>(dA[nt], dA[nt + 1], ax, b);
                            }
                    }
                    {
                        uint32_t av[3][4];
                        frag_t<3>(sa + Lay::oV, Lay::XB, ks * 16, wr * 16, av);
#pragma unroll
                        for (int nt = 0; nt < NH; nt += 2)
                            mma_cols<RBK, 3, 3, 3>(dk2[nt], dk2[nt + 1], av, sa + Lay::oS + 3 * Lay::SB, Lay::SB,
                                                   ks * 16, wc * NH + nt);
                    }
                }
                // between the products: all copies at once in front of them held up their ldmatrix
                if (ks == 0 && more)
                    raw_tokens(hi * tiles + ti + 1);
            }
        }
        for (int m = 1; m < 32; m <<= 1)
            sd += __shfl_xor_sync(0xffffffffu, sd, m);
        if (lane == 0)
            rsd[warp] = sd;
        xv[fp][ft] = xd;
        // dq's first term and its product with q; dk's two and theirs with k
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = i0 + hf * 8;
            const float e = vec[i], f = p.scale * e, fx = -vec[2 * kDeltaC + i] * e, fv = vec[kDeltaC + i];
            float dot = 0.f, kl = 0.f, rd = 0.f;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const float2 qv = pair(Lay::oQ, i, nt), kv = pair(Lay::oK, i, nt);
                float &a = dq[nt][hf * 2], &b = dq[nt][hf * 2 + 1];
                a *= f;
                b *= f;
                dot = fmaf(a, qv.x, fmaf(b, qv.y, dot));
                const float va = fv * dk2[nt][hf * 2], vb = fv * dk2[nt][hf * 2 + 1];
                kl = fmaf(va, kv.x, fmaf(vb, kv.y, kl));
                float &x = dk[nt][hf * 2], &y = dk[nt][hf * 2 + 1];
                rd = fmaf(x, kv.x, fmaf(y, kv.y, rd));
                x = fmaf(fx, x, va);
                y = fmaf(fx, y, vb);
                if constexpr (SHARED) {
                    dqt[nt][hf * 2] += a;
                    dqt[nt][hf * 2 + 1] += b;
                    dkt[nt][hf * 2] += x;
                    dkt[nt][hf * 2 + 1] += y;
                }
            }
            rd *= e;
            for (int m = 1; m < 4; m <<= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, m);
                kl += __shfl_xor_sync(0xffffffffu, kl, m);
                rd += __shfl_xor_sync(0xffffffffu, rd, m);
            }
            if ((lane & 3) == 0) {
                rowQ[wc][i] = dot;
                rowK[wc][i] = kl;
                rowR[wc][i] = rd;
            }
        }
        // k.k and q.k of the warp's rows and tokens
        float kk[4][4], qk[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                kk[n][j] = qk[n][j] = 0.f;
        if (act && wc * 2 <= wr) {
            delta_rows_product<DKP, NPI, 4>(sa + Lay::oK, sa + Lay::oK, wr * 16, wc * 32, kk);
            delta_rows_product<DKP, NPI, 4>(sa + Lay::oQ, sa + Lay::oK, wr * 16, wc * 32, qk);
        }
        __syncthreads();   // every warp is done with S^T: GP and GA take its place
        unsigned char *gp = dsm + Lay::oS, *ga = gp + NPG * kTriBytes;
        float re[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f}, ce[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int bj = wc * 2 + n / 2, jc = (n & 1) * 8 + t2;
            ce[2 * n] = ce[2 * n + 1] = 0.f;
            if (act && bj <= wr) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int i = i0 + hf * 8;
                    float vp[2], va[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {   // chosen after the arithmetic: branches took twice the time
                        const int j = bj * 16 + jc + e, x = hf * 2 + e;
                        const float D = delta_decay(ch[i] - ch[j], cl[i] - cl[j]), da = -D * dA[n][x];
                        const float pp = p.scale * D * dP[n][x], r = j < i ? kk[n][x] * da : 0.f;
                        vp[e] = j <= i ? pp : 0.f;
                        va[e] = j < i ? be[i] * da : 0.f;
                        const float E = j <= i ? fmaf(be[i], r, pp * qk[n][x]) : 0.f;
                        rb[hf] += r;
                        re[hf] += E;
                        ce[2 * n + e] += E;
                    }
                    uint32_t w[NPG];
                    const uint32_t o = tri_block(wr, bj) + tri_piece(g8 + hf * 8, n & 1) + t2 * 2;
                    split2<NPG>(vp[0], vp[1], w);
#pragma unroll
                    for (int m = 0; m < NPG; ++m)
                        *reinterpret_cast<uint32_t *>(gp + m * kTriBytes + o) = w[m];
                    split2<NPG>(va[0], va[1], w);
#pragma unroll
                    for (int m = 0; m < NPG; ++m)
                        *reinterpret_cast<uint32_t *>(ga + m * kTriBytes + o) = w[m];
                }
            }
        }
        // column sums over the eight rows of a lane's group: lane g8 ends with column pair g8 / 2, column g8 % 2
#pragma unroll
        for (int m = 4; m; m >>= 1) {
            const bool up = g8 & m;
#pragma unroll
            for (int k = 0; k < m; ++k)
                ce[k] = (up ? ce[k + m] : ce[k]) + __shfl_xor_sync(0xffffffffu, up ? ce[k] : ce[k + m], 4 * m);
        }
        colE[wr][wc * 32 + (g8 >> 1) * 8 + t2 + (g8 & 1)] = ce[0];
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
        __syncthreads();
        // lane l holds tokens 2l, 2l + 1
        if (warp == 4) {   // dc, and its sums from the end; what the last token has besides goes to all
            float dc[2], kls = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const float kl = rowK[0][i] + rowK[1][i], rd = rowR[0][i] + rowR[1][i];
                kls += kl;
                const float E = (rowE[0][i] + rowE[1][i]) - ((colE[0][i] + colE[1][i]) + (colE[2][i] + colE[3][i]));
                dc[e] = ((E + (rowQ[0][i] + rowQ[1][i])) - be[i] * rd) - kl;
            }
            float t = 0.f, sum = dc[0] + dc[1];
            for (int w = 0; w < 8; ++w)
                t += rsd[w];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                kls += __shfl_xor_sync(0xffffffffu, kls, o);
                const float u = __shfl_down_sync(0xffffffffu, sum, o);
                if (lane + o < 32)
                    sum += u;
            }
            const float last = kls + vec[kDeltaC - 1] * t;
            float after = __shfl_down_sync(0xffffffffu, sum, 1);
            after = ((lane < 31 ? after : 0.f) + dc[1]) + last;
            if (t0 + 2 * lane < q.len)
                p.dg[delta_token(p, q, t0 + 2 * lane) * p.H + h] = after + dc[0];
            if (t0 + 2 * lane + 1 < q.len)
                p.dg[delta_token(p, q, t0 + 2 * lane + 1) * p.H + h] = after;
        } else if (warp == 5) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                if (t0 + i < q.len)
                    p.dbeta[delta_token(p, q, t0 + i) * p.H + h] =
                        (((xv[0][i] + xv[1][i]) + (xv[2][i] + xv[3][i])) - (rowR[0][i] + rowR[1][i])) +
                        (rowB[0][i] + rowB[1][i]);
            }
        }
        // GP K into dq; GP^T Q, GA K, GA^T K into dk
        if (act) {
            auto &dqs = *[&] {
                if constexpr (SHARED)
                    return &dqt;
                else
                    return &dq;
            }();
            auto &dks = *[&] {
                if constexpr (SHARED)
                    return &dkt;
                else
                    return &dk;
            }();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t a[NPG][4], b[NPG][4];
                if (ks <= wr) {
                    frag_block<NPG>(smem_addr(gp) + tri_block(wr, ks), a);
                    frag_block<NPG>(smem_addr(ga) + tri_block(wr, ks), b);
#pragma unroll
                    for (int nt = 0; nt < NH; nt += 2) {
                        mma_cols<RBK, NPG, NPI, NPG>(dqs[nt], dqs[nt + 1], a, sa + Lay::oK, PBK, ks * 16,
                                                     wc * NH + nt);
                        mma_cols<RBK, NPG, NPI, NPG>(dks[nt], dks[nt + 1], b, sa + Lay::oK, PBK, ks * 16, wc * NH + nt);
                    }
                }
                if (ks >= wr && ks < nb) {
                    frag_block_t<NPG>(smem_addr(gp) + tri_block(ks, wr), a);
                    frag_block_t<NPG>(smem_addr(ga) + tri_block(ks, wr), b);
#pragma unroll
                    for (int nt = 0; nt < NH; nt += 2) {
                        mma_cols<RBK, NPG, NPI, NPG>(dks[nt], dks[nt + 1], a, sa + Lay::oQ, PBK, ks * 16, wc * NH + nt);
                        mma_cols<RBK, NPG, NPI, NPG>(dks[nt], dks[nt + 1], b, sa + Lay::oK, PBK, ks * 16, wc * NH + nt);
                    }
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
    if constexpr (SHARED) {
        store(p.dq, dqt);
        store(p.dk, dkt);
    } else {
        store(p.dq, dq);
        store(p.dk, dk);
    }
}

}  // namespace ss2d
