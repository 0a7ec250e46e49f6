// ss2d_delta.cuh -- the gated delta rule: what its kernels share, the
// token-by-token kernel, and the kernel that prepares the chunks.
//
// Per sequence and value head, state S (DK, DV), S_0 = h0, a_t = exp(g_t):
//     d_t = beta_t (v_t - a_t S_{t-1}^T k_t)
//     S_t = a_t S_{t-1} + k_t d_t^T,   o_t = scale S_t^T q_t
// (the state forgets by a, then what it holds for k_t moves towards v_t by
// beta_t).  By chunks of C = 64 tokens, with c_i = sum of g up to token i of the chunk,
// D_ij = exp(c_i - c_j) for i >= j and S the state before the chunk:
//     A  = strict lower part of beta_i D_ij k_i.k_j,   T = (I + A)^{-1}
//     Y  = V - e^c (K S),   X = beta Y,   V' = T X          (row t of V' is d_t)
//     P  = scale D_ij q_i.k_j (i >= j),   O = scale e^c (Q S) + P V'
//     S <- e^{c_last} S + K^T (e^{c_last - c} V')
// T and P of every chunk are independent of the states and come from
// delta_prep_kernel; the states are a chain over the chunks (ss2d_delta_chain.cuh).
//
// Precision.  The products run on the tensor cores with 16-bit operands and float32
// sums.  A float32 operand is split into bfloat16 parts of 8 bits each: three hold
// it exactly, and a product of two split operands is the sum of the partial products
// whose parts' indices add up to less than the number of parts kept (3: what
// is left out is below 2^-24 of the product, as a float32 rounding is).  Two parts
// hold 16 bits and leave out 2^-16 of a product.  They are used where
// only results that are rounded to 16 bits are made of them: P in every
// forward pass of 16-bit inputs, S, X, V' and T there if no last state is asked for, and
// the products with GP and GA in the gradients dq and dk of 16-bit inputs.  bfloat16
// inputs are one part: q.k needs one product and k.S three.  float16 k and q are
// operands as they are against two scaled float16 parts, 22 bits of a row's largest value,
// in the chains (see below); in the outputs of few wide heads and in the gradient kernel they are
// two bfloat16 parts, which hold them exactly.  States, sums of g (in double within a
// chunk: differences of near tokens behind a large sum keep float32
// accuracy) and everything elementwise stay float32, the exponentials on ex2.approx (2^-22).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ss2d_kernels.cuh"

namespace ss2d {

constexpr int kDeltaC = 64;         // tokens per chunk
constexpr int kDeltaMaxDK = 128;
constexpr int kDeltaMaxDV = 256;
// exp(g) of anything below is 0 in float32; a finite floor keeps sums of g finite (g = -inf forgets all)
constexpr float kDeltaGFloor = -200.f;
constexpr int kDeltaVec = 5 * kDeltaC;   // floats of `vec` per (slot, head)

struct DeltaParams {
    const void *q, *k, *v;         // token rows: HK x DK (q, k), H x DV (v)
    long long qs, ks, vs;          // values between tokens
    const float *g, *beta;         // (tokens, H)
    const int *cu;                 // first token of each sequence (nseq + 1), or null: nseq sequences of L
    const float *h0;               // (nseq, H, DK, DV) or null
    float *h_last;                 // (nseq, H, DK, DV) or null
    void *o;                       // (tokens, H, DV)
    long long T;                   // tokens
    int nseq, L, HK, H, DK, DV;
    int reverse;                   // a sequence is read from its last token to its first
    float scale;
    // step: states and the row of the pool that each sequence uses
    float *pool;
    const int *slots;
    long long npool;
    // scratch of the chunks
    int NC;                        // chunk slots per sequence (cu null)
    long long nslots;
    void *kp, *qp;                 // bf16 parts of k and q per (slot, key head): [NPI][64][DKP]; null: nobody reads them
    void *Tp, *Pp;                 // bf16 parts of T and P per (slot, head), packed blocks
    float *vec;                    // per (slot, head): e^c, e^{c_last - c}, beta, c log2(e) and what it lacks (64 each)
    // segments of a long chain: SC chunks each (0: none)
    int SC;
    float *Ns, *dNs;               // S^T at a segment's end from zero, dS^T at its start: [DV][DKP] per (segment, head)
    void *Ms;                      // three bf16 parts of its transition: [DKP][DKP] per (segment, head)
    float *Sin, *dSin;             // S^T a segment starts from, dS^T it ends with
    // backward
    const void *dout;              // gradient of o
    const float *dh_last;
    float *dh0;
    void *dq, *dk, *dv;
    float *dg, *dbeta;
    float *Sx, *dSx;               // S before, dS after each chunk: [DV][DKP] per (slot, head)
    float *Vx, *dXx;               // V', dX: [DV][64] per (slot, head)
};

struct DeltaSeq {
    long long start;
    int len;
};
// sequence s, held inside the tokens whatever cu says
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaParams &p, int s)
{
    if (!p.cu)
        return {(long long)s * p.L, p.L};
    long long a = p.cu[s], b = p.cu[s + 1];
    a = a < 0 ? 0 : (a > p.T ? p.T : a);
    b = b < a ? a : (b > p.T ? p.T : b);
    return {a, (int)(b - a)};
}
// first chunk slot of a sequence: ceil(len / 64) slots from here never reach
// the next sequence's, nor floor(T / 64) + nseq
__device__ __forceinline__ long long delta_slot0(const DeltaParams &p, int s, const DeltaSeq &q)
{
    return p.cu ? q.start / kDeltaC + s : (long long)s * p.NC;
}
// the (sequence, chunk) of a slot; false: the slot holds none
__device__ __forceinline__ bool delta_slot(const DeltaParams &p, long long slot, int &s, DeltaSeq &q, int &c)
{
    if (!p.cu) {
        s = (int)(slot / p.NC);
        c = (int)(slot - (long long)s * p.NC);
        q = delta_seq(p, s);
    } else {
        int lo = 0, hi = p.nseq - 1;   // the last sequence that starts at or before the slot
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            const DeltaSeq t = delta_seq(p, m);
            if (delta_slot0(p, m, t) <= slot)
                lo = m;
            else
                hi = m - 1;
        }
        s = lo;
        q = delta_seq(p, s);
        const long long d = slot - delta_slot0(p, s, q);
        if (d < 0 || d * kDeltaC >= q.len)
            return false;
        c = (int)d;
    }
    return (long long)c * kDeltaC < q.len;
}
// token that step t of a sequence reads
__device__ __forceinline__ long long delta_token(const DeltaParams &p, const DeltaSeq &q, int t)
{
    return q.start + (p.reverse ? q.len - 1 - t : t);
}

// Segments.  A segment's slot is found like a chunk's: ceil(chunks / SC) slots from
// here never reach the next sequence's.
__device__ __forceinline__ long long delta_seg0(const DeltaParams &p, int s, const DeltaSeq &q)
{
    return p.cu ? delta_slot0(p, s, q) / p.SC + s : (long long)s * ((p.NC + p.SC - 1) / p.SC);
}
// the sequence and chunks [c0, c1) of a chain's unit: a segment, or a whole sequence; false: the unit holds none
__device__ __forceinline__ bool delta_unit(const DeltaParams &p, long long unit, int &s, DeltaSeq &q, int &c0, int &c1)
{
    if (!p.SC) {
        s = (int)unit;
        q = delta_seq(p, s);
        c0 = 0;
        c1 = (q.len + kDeltaC - 1) / kDeltaC;
        return true;
    }
    int seg;
    if (!p.cu) {
        const int n = (p.NC + p.SC - 1) / p.SC;
        s = (int)(unit / n);
        seg = (int)(unit - (long long)s * n);
        q = delta_seq(p, s);
    } else {
        int lo = 0, hi = p.nseq - 1;
        while (lo < hi) {
            const int m = (lo + hi + 1) >> 1;
            if (delta_seg0(p, m, delta_seq(p, m)) <= unit)
                lo = m;
            else
                hi = m - 1;
        }
        s = lo;
        q = delta_seq(p, s);
        const long long d = unit - delta_seg0(p, s, q);
        if (d < 0 || d > q.len / kDeltaC)
            return false;
        seg = (int)d;
    }
    const int nc = (q.len + kDeltaC - 1) / kDeltaC;
    c0 = seg * p.SC;
    c1 = min(c0 + p.SC, nc);
    return c0 < c1;
}

// ---- bf16 parts ------------------------------------------------------------
template <typename T>
struct DeltaParts;   // parts that hold a value of the type exactly
template <>
struct DeltaParts<__nv_bfloat16> {
    static constexpr int n = 1;
};
template <>
struct DeltaParts<__half> {
    static constexpr int n = 2;
};
template <>
struct DeltaParts<float> {
    static constexpr int n = 3;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// the first N bf16 parts of (x, y), packed
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&o)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        o[i] = pack_bf16(x, y);
        if (i + 1 < N) {
            x -= __uint_as_float(o[i] << 16);
            y -= __uint_as_float(o[i] & 0xffff0000u);
        }
    }
}

// ---- tensor-core and shared-memory pieces ------------------------------------
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(on ? 16u : 0u)
                 : "memory");
}
// byte offset of the 16-byte piece `pc` of row `r` in a tile of rows of RB
// bytes (a multiple of 128): pieces of eight neighbouring rows fall into
// eight different bank groups, for ldmatrix by rows and by columns
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int pc)
{
    return (uint32_t)(r * RB + ((pc ^ (r & 7)) << 4));
}
// A lower triangular 64 x 64 bf16 part as its ten 16 x 16 blocks (bi >= bj), 512
// bytes each, rows of 32 bytes whose two pieces change places every four rows, so
// that eight rows of a piece fall into eight different bank groups.
constexpr int kTriBytes = 10 * 512;
__device__ __forceinline__ uint32_t tri_block(int bi, int bj) { return (uint32_t)((bi * (bi + 1) / 2 + bj) * 512); }
__device__ __forceinline__ uint32_t tri_piece(int r, int pc) { return (uint32_t)(r * 32 + ((pc ^ (r >> 2 & 1)) << 4)); }
// C fragments of two neighbouring 8-column tiles as the A operand of the 16
// columns they span, in N parts
template <int N>
__device__ __forceinline__ void frag_a(const float (&c0)[4], const float (&c1)[4], uint32_t (&a)[N][4])
{
    uint32_t t[N];
    split2<N>(c0[0], c0[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i)
        a[i][0] = t[i];
    split2<N>(c0[2], c0[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i)
        a[i][1] = t[i];
    split2<N>(c1[0], c1[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i)
        a[i][2] = t[i];
    split2<N>(c1[2], c1[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i)
        a[i][3] = t[i];
}

// c0, c1 (16 x 8 each) += A parts (NA) times B parts (NB), the products whose
// part indices add up to less than KEEP.  The tensor cores' sums truncate
// (each accumulation loses up to 2^-23 of the sum, always downwards), so
// three-part products are summed from zero, smallest parts first, and added to
// the result by a rounding float32 addition: measured on the float32 backward
// (32 x 64 heads, 1500 tokens) the gradients are 2.8e-7 off instead of 3.8e-6.  The additions
// issue in the tensor pipe's shadow.  A product of two exact operands
// is one accumulation for 16 columns, and goes into the result as it is.
template <int NA, int NB, int KEEP>
__device__ __forceinline__ void mma_parts(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                          const uint32_t (&b)[NB][4])
{
    if constexpr (KEEP == 3 && NA * NB > 1) {
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sum = KEEP - 1; sum >= 0; --sum)
#pragma unroll
            for (int m = 0; m < NB; ++m)
                if (sum - m >= 0 && sum - m < NA) {
                    mma16816(d0, a[sum - m], b[m][0], b[m][1]);
                    mma16816(d1, a[sum - m], b[m][2], b[m][3]);
                }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c0[j] += d0[j];
            c1[j] += d1[j];
        }
    } else {
#pragma unroll
        for (int m = 0; m < NB; ++m)
#pragma unroll
            for (int n = 0; n < NA; ++n)
                if (n + m < KEEP) {
                    mma16816(c0, a[n], b[m][0], b[m][1]);
                    mma16816(c1, a[n], b[m][2], b[m][3]);
                }
    }
}

// B from rows of a [n][k] tile: B element (k, n) is row n, column k
template <int RB, int N>
__device__ __forceinline__ void frag_rows(uint32_t tile, int part, int row, int piece, uint32_t (&b)[N][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 0; m < N; ++m)
        ldsm4(tile + m * part + swz<RB>(row + (lane & 7) + (lane >> 4) * 8, piece + (lane >> 3 & 1)), b[m]);
}
template <int RB, int NA, int NB, int KEEP>
__device__ __forceinline__ void mma_rows(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4], uint32_t tile,
                                         int part, int row, int piece)
{
    constexpr int NL = NB < KEEP ? NB : KEEP;
    uint32_t b[NL][4];
    frag_rows<RB, NL>(tile, part, row, piece, b);
    mma_parts<NA, NL, KEEP>(c0, c1, a, b);
}
// B from a [k][n] tile: rows k, columns n
template <int RB, int N>
__device__ __forceinline__ void frag_cols(uint32_t tile, int part, int row, int piece, uint32_t (&b)[N][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 0; m < N; ++m)
        ldsm4t(tile + m * part + swz<RB>(row + (lane & 15), piece + (lane >> 4)), b[m]);
}
template <int RB, int NA, int NB, int KEEP>
__device__ __forceinline__ void mma_cols(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4], uint32_t tile,
                                         int part, int row, int piece)
{
    constexpr int NL = NB < KEEP ? NB : KEEP;
    uint32_t b[NL][4];
    frag_cols<RB, NL>(tile, part, row, piece, b);
    mma_parts<NA, NL, KEEP>(c0, c1, a, b);
}

// ---- float16 inputs as they are -----------------------------------------------
// K and Q of float16 calls are one exact float16 operand each, where bfloat16 parts would
// be two; what multiplies them is split into two float16 parts (22 bits) after
// scaling each row (a column of DV) by the power of two that brings its largest value into
// 2^13 .. 2^14: two products instead of five, and half the shared memory.  A value
// smaller than its row's largest by 2^16 and more keeps fewer bits, but none is off by
// more than 2^-38 of the largest.  16384 packed tokens, 16 heads of 128: outputs 510 -> 380 us
// (358 with one scale for a warp, where a small column next to a large one lost bits), preparation 127 -> 66.
struct HalfScale {
    float up[2], down[2];   // of the lane's rows
};
template <int N>
__device__ __forceinline__ HalfScale half_scale(const float (&v)[N][4])
{
    HalfScale s;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float m = 0.f;   // a NaN is passed over here and stays one in its part
#pragma unroll
        for (int n = 0; n < N; ++n)
            m = fmaxf(m, fmaxf(fabsf(v[n][2 * r]), fabsf(v[n][2 * r + 1])));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t e = max(__float_as_uint(m) >> 23, 14u);
        s.up[r] = __uint_as_float((267u - e) << 23);
        s.down[r] = __uint_as_float((e - 13u) << 23);
    }
    return s;
}
__device__ __forceinline__ void half_split(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ void half_frag(const float (&c0)[4], const float (&c1)[4], const float (&up)[2],
                                          uint32_t (&a)[2][4])
{
    half_split(c0[0] * up[0], c0[1] * up[0], a[0][0], a[1][0]);
    half_split(c0[2] * up[1], c0[3] * up[1], a[0][1], a[1][1]);
    half_split(c1[0] * up[0], c1[1] * up[0], a[0][2], a[1][2]);
    half_split(c1[2] * up[1], c1[3] * up[1], a[0][3], a[1][3]);
}
__device__ __forceinline__ void mma16816h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c0, c1 += A B: FROM0 summed from zero and joined by a rounding addition that takes the scale off (see mma_parts),
// otherwise in the scaled sum itself
template <bool FROM0>
__device__ __forceinline__ void mma_half(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[2][4],
                                         const uint32_t (&b)[4], const float (&down)[2])
{
    if constexpr (FROM0) {
        float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 1; n >= 0; --n) {
            mma16816h(d0, a[n], b[0], b[1]);
            mma16816h(d1, a[n], b[2], b[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c0[j] = fmaf(d0[j], down[j >> 1], c0[j]);
            c1[j] = fmaf(d1[j], down[j >> 1], c1[j]);
        }
    } else {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma16816h(c0, a[n], b[0], b[1]);
            mma16816h(c1, a[n], b[2], b[3]);
        }
    }
}

// B from a 16 x 16 block of packed parts: its rows are n (columns k), or its rows are k (columns n)
template <int NA, int NB, int KEEP>
__device__ __forceinline__ void mma_block_rows(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                               uint32_t block)
{
    const int lane = threadIdx.x & 31;
    uint32_t b[NB][4];
#pragma unroll
    for (int m = 0; m < NB; ++m)
        ldsm4(block + m * kTriBytes + tri_piece((lane & 7) + (lane >> 4) * 8, lane >> 3 & 1), b[m]);
    mma_parts<NA, NB, KEEP>(c0, c1, a, b);
}
template <int NA, int NB, int KEEP>
__device__ __forceinline__ void mma_block_cols(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                               uint32_t block)
{
    const int lane = threadIdx.x & 31;
    uint32_t b[NB][4];
#pragma unroll
    for (int m = 0; m < NB; ++m)
        ldsm4t(block + m * kTriBytes + tri_piece(lane & 15, lane >> 4), b[m]);
    mma_parts<NA, NB, KEEP>(c0, c1, a, b);
}
// A from a packed block, rows m (columns k), or transposed: rows k (columns m)
template <int N>
__device__ __forceinline__ void frag_block(uint32_t block, uint32_t (&a)[N][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < N; ++n)
        ldsm4(block + n * kTriBytes + tri_piece(lane & 15, lane >> 4), a[n]);
}
template <int N>
__device__ __forceinline__ void frag_block_t(uint32_t block, uint32_t (&a)[N][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < N; ++n)
        ldsm4t(block + n * kTriBytes + tri_piece((lane & 7) + (lane >> 4) * 8, lane >> 3 & 1), a[n]);
}
// A fragment (rows m0.., columns k0..) of a tile stored [k][m] in rows of 128 bytes
template <int N>
__device__ __forceinline__ void frag_t(uint32_t tile, int part, int k0, int m0, uint32_t (&a)[N][4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < N; ++n)
        ldsm4t(tile + n * part + swz<128>(k0 + (lane & 7) + (lane >> 4) * 8, m0 / 8 + (lane >> 3 & 1)), a[n]);
}

// ---- token by token ----------------------------------------------------------
// The recurrence as it stands, for sequences of a few tokens and for one token
// of many sequences with the states updated in place.  A CTA holds DVT columns
// of one state in registers, thread (row group rg, four columns): k.S and q.S
// need one pass over the rows and one sum over the row groups, since
// o = scale (a q.S + (q.k) d).  Bound by reading and writing the states
// once: DK * DVT * 8 bytes per CTA, in 16-byte pieces along DV.
constexpr int kRecurThreads = 256;

// ROWS: rows of the state per thread
template <typename Tin, int ROWS>
__global__ void __launch_bounds__(kRecurThreads, 4) delta_recur_kernel(const DeltaParams p, int DVT)
{
    __shared__ float sk[kDeltaMaxDK], sq[kDeltaMaxDK];
    __shared__ __align__(16) float red[2][kRecurThreads][4];
    __shared__ float sqk;
    const int tid = threadIdx.x;
    const int nv4 = DVT / 4, RG = kRecurThreads / nv4;
    const int c4 = tid % nv4, rg = tid / nv4;
    const int h = blockIdx.y, hk = h / (p.H / p.HK);
    const int dv0 = blockIdx.x * DVT + c4 * 4;
    const bool on = rg < RG && dv0 < p.DV;
    for (long long sn = blockIdx.z; sn < p.nseq; sn += gridDim.z) {
        const DeltaSeq q = delta_seq(p, (int)sn);
        long long si = sn;   // state read and written
        bool live = true;
        if (p.pool && p.slots) {
            si = p.slots[sn];
            live = si >= 0 && si < p.npool;
            bool dup = false;   // the first sequence of a slot has it
            for (long long i = tid; i < sn; i += kRecurThreads)
                dup |= p.slots[i] == (int)si;
            live = !__syncthreads_or(dup) && live;
        }
        const long long srow = (si * p.H + h) * p.DK;
        float4 S[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = rg + i * RG;
            S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float *src = p.pool ? p.pool : p.h0;
            if (on && live && r < p.DK && src)
                S[i] = *reinterpret_cast<const float4 *>(src + (srow + r) * p.DV + dv0);
        }
        for (int t = 0; t < q.len; ++t) {
            const long long tok = delta_token(p, q, t);
            __syncthreads();
            if (tid < 2 * kDeltaMaxDK) {
                const int i = tid % kDeltaMaxDK;
                const Tin *src = tid < kDeltaMaxDK ? static_cast<const Tin *>(p.k) + tok * p.ks
                                                   : static_cast<const Tin *>(p.q) + tok * p.qs;
                const float v = live && i < p.DK ? to_f32(src[(long long)hk * p.DK + i]) : 0.f;
                (tid < kDeltaMaxDK ? sk : sq)[i] = v;
            }
            __syncthreads();
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int r = rg + i * RG;
                if (r < p.DK) {
                    const float kv = sk[r], qv = sq[r];
                    a.x = fmaf(kv, S[i].x, a.x);
                    a.y = fmaf(kv, S[i].y, a.y);
                    a.z = fmaf(kv, S[i].z, a.z);
                    a.w = fmaf(kv, S[i].w, a.w);
                    b.x = fmaf(qv, S[i].x, b.x);
                    b.y = fmaf(qv, S[i].y, b.y);
                    b.z = fmaf(qv, S[i].z, b.z);
                    b.w = fmaf(qv, S[i].w, b.w);
                }
            }
            *reinterpret_cast<float4 *>(red[0][tid]) = a;
            *reinterpret_cast<float4 *>(red[1][tid]) = b;
            if (tid < 32) {
                float s = 0.f;
                for (int i = tid; i < p.DK; i += 32)
                    s = fmaf(sk[i], sq[i], s);
                for (int m = 16; m; m >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, m);
                if (tid == 0)
                    sqk = s;
            }
            __syncthreads();
            a = b = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < RG; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(red[0][i * nv4 + c4]);
                const float4 y = *reinterpret_cast<const float4 *>(red[1][i * nv4 + c4]);
                a.x += x.x;
                a.y += x.y;
                a.z += x.z;
                a.w += x.w;
                b.x += y.x;
                b.y += y.y;
                b.z += y.z;
                b.w += y.w;
            }
            if (on && live) {
                const float gv = p.g[tok * p.H + h], be = p.beta[tok * p.H + h];
                const float al = expf(gv < kDeltaGFloor ? kDeltaGFloor : gv);
                const Tin *vr = static_cast<const Tin *>(p.v) + tok * p.vs + (long long)h * p.DV + dv0;
                float4 d;
                d.x = be * (to_f32(vr[0]) - al * a.x);
                d.y = be * (to_f32(vr[1]) - al * a.y);
                d.z = be * (to_f32(vr[2]) - al * a.z);
                d.w = be * (to_f32(vr[3]) - al * a.w);
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    const int r = rg + i * RG;
                    if (r < p.DK) {
                        const float kv = sk[r];
                        S[i].x = fmaf(kv, d.x, al * S[i].x);
                        S[i].y = fmaf(kv, d.y, al * S[i].y);
                        S[i].z = fmaf(kv, d.z, al * S[i].z);
                        S[i].w = fmaf(kv, d.w, al * S[i].w);
                    }
                }
                if (rg == 0) {
                    const float w[4] = {p.scale * fmaf(sqk, d.x, al * b.x), p.scale * fmaf(sqk, d.y, al * b.y),
                                        p.scale * fmaf(sqk, d.z, al * b.z), p.scale * fmaf(sqk, d.w, al * b.w)};
                    Tin *orow = static_cast<Tin *>(p.o) + (tok * p.H + h) * p.DV + dv0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (std::is_same_v<Tin, float>)
                            orow[j] = w[j];
                        else if constexpr (std::is_same_v<Tin, __half>)
                            orow[j] = __float2half_rn(w[j]);
                        else
                            orow[j] = __float2bfloat16_rn(w[j]);
                    }
                }
            } else if (on && rg == 0) {
                Tin *orow = static_cast<Tin *>(p.o) + (tok * p.H + h) * p.DV + dv0;
                for (int j = 0; j < 4; ++j)
                    orow[j] = Tin(0.f);
            }
        }
        float *dst = p.pool ? p.pool : p.h_last;
        if (on && live && dst) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int r = rg + i * RG;
                if (r < p.DK)
                    *reinterpret_cast<float4 *>(dst + (srow + r) * p.DV + dv0) = S[i];
            }
        }
        __syncthreads();
    }
}

// ---- chunk preparation ---------------------------------------------------------
// Per (slot, key head): K K^T and Q K^T on the tensor cores (K and Q as they are in
// 16 bits; in bf16 parts, with scratch copies, where the chain reads them so), and for
// each value head of the group T and P in bf16 parts and the chunk's e^c,
// e^{c_last - c}, beta, c.  Steps past the sequence's end have k = q = 0, g = 0,
// beta = 0: they leave the state as it is.
//
// 4 warps share the ten 16 x 16 blocks of the products.  T = (I + A)^{-1} by such
// blocks: warp w inverts block (w, w) by forward substitution in
// float32 (lane j its column j), then has the blocks below it,
//     T_iw = -T_ii sum_{w <= m < i} A_im T_mw,   i = w + 1 .. 3,
// as tensor-core products of bf16 parts, transposed like the chain's, so that
// each result is the next product's A operand.  (One thread per column of the
// whole 64 x 64 substitution, the first form, waited on 64 dependent rows: 363 us
// for 6144 chunks of 64 x 64 heads, 74 now with two parts, 89 with three.)  T and P leave through shared memory in
// 16-byte pieces, the blocks above the diagonal not at all.
constexpr int kPrepThreads = 128;

template <int DKP, int NPI, int NPT, int NPP>
struct PrepLayout {
    static constexpr int oT = NPT * kTriBytes;                 // T; A before it
    static constexpr int oP = oT + NPT * kTriBytes;            // a block of P for each warp
    static constexpr int oD = oP + 4 * NPP * 512;
    static constexpr int head = oD + 4 * 16 * 20 * 4;          // diagonal blocks of A, rows of 20 floats
    static constexpr int tiles = 2 * NPI * kDeltaC * DKP * 2;  // K and Q, read before the heads
    static constexpr int bytes = tiles > head ? tiles : head;
};

// NPI x 64 x DKP bf16 parts of the token rows of q or k into a swizzled tile: by
// asynchronous copies where the input is its own part (the caller waits for them)
template <typename Tin, int DKP, int NPI, int NT>
__device__ __forceinline__ void delta_stage_parts(const DeltaParams &p, const void *base, long long ts, int hk,
                                                  const DeltaSeq &q, int t0, unsigned char *tile)
{
    constexpr int RB = DKP * 2, PPR = DKP / 8;
    static_assert(kDeltaC * PPR % NT == 0, "whole rounds");
    const Tin *src = static_cast<const Tin *>(base) + (long long)hk * p.DK;
#pragma unroll 4
    for (int k = 0; k < kDeltaC * PPR / NT; ++k) {
        const int i = k * NT + threadIdx.x, r = i / PPR, pc = i % PPR;
        const bool in = t0 + r < q.len && pc * 8 < p.DK;
        const Tin *row = src + delta_token(p, q, in ? t0 + r : 0) * ts + (in ? pc * 8 : 0);
        if constexpr (NPI == 1) {
            cp16(smem_addr(tile) + swz<RB>(r, pc), row, in);
        } else {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = 0.f;
            if (in) {
                if constexpr (sizeof(Tin) == 2) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(row);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = half_bits_to_f32<Tin>(w[j] & 0xffffu);
                        v[2 * j + 1] = half_bits_to_f32<Tin>(w[j] >> 16);
                    }
                } else {
                    const float4 f0 = *reinterpret_cast<const float4 *>(row);
                    const float4 f1 = *reinterpret_cast<const float4 *>(row + 4);
                    v[0] = f0.x;
                    v[1] = f0.y;
                    v[2] = f0.z;
                    v[3] = f0.w;
                    v[4] = f1.x;
                    v[5] = f1.y;
                    v[6] = f1.z;
                    v[7] = f1.w;
                }
            }
            uint32_t w[4][NPI];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                split2<NPI>(v[2 * j], v[2 * j + 1], w[j]);
#pragma unroll
            for (int n = 0; n < NPI; ++n)
                *reinterpret_cast<uint4 *>(tile + n * kDeltaC * RB + swz<RB>(r, pc)) =
                    make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
        }
    }
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

// acc (16 rows x 8 NT columns of a warp) += rows r0.. of tile A times rows n0.. of tile B, transposed: sums over DKP
template <int DKP, int NPI, int NT, bool HALF = false>
__device__ __forceinline__ void delta_rows_product(uint32_t A, uint32_t B, int r0, int n0, float (&acc)[NT][4])
{
    constexpr int RB = DKP * 2, PB = kDeltaC * RB;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int ks = 0; ks < DKP / 16; ++ks) {
        uint32_t a[NPI][4];
#pragma unroll
        for (int n = 0; n < NPI; ++n)
            ldsm4(A + n * PB + swz<RB>(r0 + (lane & 15), ks * 2 + (lane >> 4)), a[n]);
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
            uint32_t b[NPI][4];
#pragma unroll
            for (int m = 0; m < NPI; ++m)
                ldsm4(B + m * PB + swz<RB>(n0 + nt * 8 + (lane & 7) + (lane >> 4) * 8, ks * 2 + (lane >> 3 & 1)),
                      b[m]);
            if constexpr (HALF) {   // float16 as it is
                mma16816h(acc[nt], a[0], b[0][0], b[0][1]);
                mma16816h(acc[nt + 1], a[0], b[0][2], b[0][3]);
            } else {
                mma_parts<NPI, NPI, 3>(acc[nt], acc[nt + 1], a, b);
            }
        }
    }
}

// e^x of a sum of g kept as c log2(e): a float and what it lacks, so that differences of
// near tokens behind a large sum are exact to float32
__device__ __forceinline__ float delta_decay(float h, float l) { return mufu_ex2(h + l); }

// c log2(e) (as a float and what it lacks) and beta of one head's chunk, by one warp: lane l holds tokens 2l, 2l + 1
__device__ __forceinline__ void delta_decays(const DeltaParams &p, const DeltaSeq &q, int t0, int h, float *ch,
                                             float *cl, float *be)
{
    const int lane = threadIdx.x & 31;
    double v[2];
    float b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = t0 + 2 * lane + j;
        float gv = 0.f;
        b[j] = 0.f;
        if (t < q.len) {
            const long long i = delta_token(p, q, t) * p.H + h;
            gv = p.g[i];
            gv = gv < kDeltaGFloor ? kDeltaGFloor : gv;   // a NaN stays one
            b[j] = p.beta[i];
        }
        v[j] = (double)gv * 1.4426950408889634;
    }
    double s = v[0] + v[1];
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += u;
    }
    const double c1 = s, c0 = s - v[1];
    ch[2 * lane] = (float)c0;
    cl[2 * lane] = (float)(c0 - (double)(float)c0);
    ch[2 * lane + 1] = (float)c1;
    cl[2 * lane + 1] = (float)(c1 - (double)(float)c1);
    be[2 * lane] = b[0];
    be[2 * lane + 1] = b[1];
}

// NPT parts of T, NPP of P are written; PARTS: k and q are split into bf16 parts, and copied where they are read as such
template <typename Tin, int DKP, int NPT, int NPP, bool PARTS>
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prep_kernel(const DeltaParams p)
{
    constexpr int NPI = PARTS ? DeltaParts<Tin>::n : 1, RB = DKP * 2, PB = kDeltaC * RB;
    constexpr bool HALF = !PARTS && std::is_same_v<Tin, __half>;
    using Lay = PrepLayout<DKP, NPI, NPT, NPP>;
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ float ch[kDeltaC], cl[kDeltaC], be[kDeltaC];
    int s, c;
    DeltaSeq q;
    if (!delta_slot(p, blockIdx.x, s, q, c))
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hk = blockIdx.y, G = p.H / p.HK, t0 = c * kDeltaC;
    unsigned char *kt = dsm, *qt = dsm + NPI * PB;
    delta_stage_parts<Tin, DKP, NPI, kPrepThreads>(p, p.k, p.ks, hk, q, t0, kt);
    delta_stage_parts<Tin, DKP, NPI, kPrepThreads>(p, p.q, p.qs, hk, q, t0, qt);
    if (warp == 3)
        delta_decays(p, q, t0, hk * G, ch, cl, be);
    cp_wait();
    __syncthreads();
    if constexpr (PARTS) {   // scratch copies, rows in order (not swizzled)
        const long long base = ((long long)blockIdx.x * p.HK + hk) * NPI * PB;
        for (int i = tid; i < NPI * kDeltaC * (DKP / 8); i += kPrepThreads) {
            const int r = i / (DKP / 8), pc = i % (DKP / 8);   // r counts the parts' rows
            const uint32_t so = (uint32_t)(r / kDeltaC) * PB + swz<RB>(r % kDeltaC, pc);
            *reinterpret_cast<uint4 *>(static_cast<char *>(p.kp) + base + (long long)i * 16) =
                *reinterpret_cast<const uint4 *>(kt + so);
            *reinterpret_cast<uint4 *>(static_cast<char *>(p.qp) + base + (long long)i * 16) =
                *reinterpret_cast<const uint4 *>(qt + so);
        }
    }
    // the ten blocks of the lower triangle, two or three to a warp: 00 30 31, 10 11 32, 20 21, 22 33
    constexpr int MB = 3;
    const int nblk = warp < 2 ? 3 : 2;
    const uint32_t blocks = warp == 0 ? 0x313000u : warp == 1 ? 0x321110u : warp == 2 ? 0x2120u : 0x3322u;
    auto bi = [&](int n) { return (int)(blocks >> (8 * n + 4) & 15u); };
    auto bj = [&](int n) { return (int)(blocks >> (8 * n) & 15u); };
    float kk[MB][2][4], qk[MB][2][4];
#pragma unroll
    for (int n = 0; n < MB; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            kk[n][0][j] = kk[n][1][j] = qk[n][0][j] = qk[n][1][j] = 0.f;
        if (n < nblk) {
            delta_rows_product<DKP, NPI, 2, HALF>(smem_addr(kt), smem_addr(kt), bi(n) * 16, bj(n) * 16, kk[n]);
            delta_rows_product<DKP, NPI, 2, HALF>(smem_addr(qt), smem_addr(kt), bi(n) * 16, bj(n) * 16, qk[n]);
        }
    }
    const uint32_t sA = smem_addr(dsm), sX = sA + Lay::oT;
    unsigned char *pw = dsm + Lay::oP + warp * NPP * 512;   // the warp's block of P
    float *dg = reinterpret_cast<float *>(dsm + Lay::oD);   // [4][16][20]
    const int nb = (min(q.len - t0, kDeltaC) + 15) / 16;    // 16-token blocks that hold tokens
    // a block of N parts, `from` bytes apart, to the block's place in a head's scratch, by one warp
    auto leave = [&](void *dst, long long sh, int N, int I, int J, const unsigned char *src, int from) {
        char *d = static_cast<char *>(dst) + sh * N * kTriBytes + tri_block(I, J) + lane * 16;
        for (int m = 0; m < N; ++m)
            *reinterpret_cast<uint4 *>(d + m * kTriBytes) = *reinterpret_cast<const uint4 *>(src + m * from + lane * 16);
    };
    for (int hi = 0; hi < G; ++hi) {
        const int h = hk * G + hi;
        const long long sh = (long long)blockIdx.x * p.H + h;
        __syncthreads();   // the tiles (or the last head's T) are read, the decays are here
        if (tid < kDeltaC) {
            float *vec = p.vec + sh * kDeltaVec;
            vec[tid] = delta_decay(ch[tid], cl[tid]);
            vec[kDeltaC + tid] = delta_decay(ch[kDeltaC - 1] - ch[tid], cl[kDeltaC - 1] - cl[tid]);
            vec[2 * kDeltaC + tid] = be[tid];
            vec[3 * kDeltaC + tid] = ch[tid];
            vec[4 * kDeltaC + tid] = cl[tid];
        }
        const int ir = lane >> 2, jr = (lane & 3) * 2;   // row and first column of a lane in an 8 x 8 tile
#pragma unroll
        for (int n = 0; n < MB; ++n) {
            if (n >= nblk)
                continue;
            const int I = bi(n), J = bj(n);
            const bool diag = I == J;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = ir + hf * 8;
                const float hi_ = ch[I * 16 + i], lo_ = cl[I * 16 + i], bi_ = be[I * 16 + i];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int j = t * 8 + jr;
                    const float2 hj = *reinterpret_cast<const float2 *>(ch + J * 16 + j);
                    const float2 lj = *reinterpret_cast<const float2 *>(cl + J * 16 + j);
                    float D0 = delta_decay(hi_ - hj.x, lo_ - lj.x), D1 = delta_decay(hi_ - hj.y, lo_ - lj.y);
                    if (diag) {   // above the diagonal the exponent is positive: dropped, not multiplied by zero
                        D0 = j <= i ? D0 : 0.f;
                        D1 = j < i ? D1 : 0.f;
                    }
                    const float k0 = kk[n][t][hf * 2], k1 = kk[n][t][hf * 2 + 1];
                    const float q0 = qk[n][t][hf * 2], q1 = qk[n][t][hf * 2 + 1];
                    const bool on0 = !diag || j <= i, on1 = !diag || j < i;
                    const uint32_t in = tri_piece(i, t) + (lane & 3) * 4, o = tri_block(I, J) + in;
                    uint32_t w[NPP], u[NPT];
                    split2<NPP>(on0 ? p.scale * D0 * q0 : 0.f, on1 ? p.scale * D1 * q1 : 0.f, w);
#pragma unroll
                    for (int m = 0; m < NPP; ++m)
                        *reinterpret_cast<uint32_t *>(pw + m * 512 + in) = w[m];
                    if (!diag) {
                        split2<NPT>(bi_ * D0 * k0, bi_ * D1 * k1, u);
#pragma unroll
                        for (int m = 0; m < NPT; ++m)
                            *reinterpret_cast<uint32_t *>(dsm + m * kTriBytes + o) = u[m];
                    } else {
                        *reinterpret_cast<float2 *>(dg + ((I * 16 + i) * 20 + j)) =
                            make_float2(j < i ? bi_ * D0 * k0 : 0.f, j + 1 < i ? bi_ * D1 * k1 : 0.f);
                    }
                }
            }
            __syncwarp();
            leave(p.Pp, sh, NPP, I, J, pw, 512);
            __syncwarp();
        }
        __syncthreads();   // A and its diagonal blocks are here
        // column j = lane of the diagonal block's inverse
        float col[16];
        if (lane < 16) {
            const float *a = dg + warp * 16 * 20;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a0 = 0.f, a1 = 0.f;
#pragma unroll
                for (int m = 0; m < i; m += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(a + i * 20 + m);
                    a0 = fmaf(w.x, col[m], a0);
                    if (m + 1 < i)
                        a1 = fmaf(w.y, col[m + 1], a1);
                    if (m + 2 < i)
                        a0 = fmaf(w.z, col[m + 2], a0);
                    if (m + 3 < i)
                        a1 = fmaf(w.w, col[m + 3], a1);
                }
                col[i] = (i == lane ? 1.f : 0.f) - (a0 + a1);   // zero above the diagonal by itself
            }
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x = col[i];
                unsigned char *o = dsm + Lay::oT + tri_block(warp, warp) + tri_piece(i, lane >> 3) + (lane & 7) * 2;
#pragma unroll
                for (int m = 0; m < NPT; ++m) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(x);
                    *reinterpret_cast<__nv_bfloat16 *>(o + m * kTriBytes) = b;
                    x -= __bfloat162float(b);
                }
            }
        }
        __syncthreads();
        if (warp == 3 && hi + 1 < G)   // the next head's decays, by the warp that has no column of blocks
            delta_decays(p, q, t0, h + 1, ch, cl, be);
        for (int i = warp + 1; i < 4; ++i) {
            float w0[4] = {0.f, 0.f, 0.f, 0.f}, w1[4] = {0.f, 0.f, 0.f, 0.f}, u0[4] = {0.f, 0.f, 0.f, 0.f},
                  u1[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t a[NPT][4];
            if (i < nb) {   // blocks of no token have A = 0, and T = 0
                for (int m = warp; m < i; ++m) {
                    frag_block_t<NPT>(sX + tri_block(m, warp), a);
                    mma_block_rows<NPT, NPT, NPT>(w0, w1, a, sA + tri_block(i, m));
                }
                frag_a<NPT>(w0, w1, a);
                mma_block_rows<NPT, NPT, NPT>(u0, u1, a, sX + tri_block(i, i));
            }
            uint32_t o[4][NPT];
            split2<NPT>(-u0[0], -u0[1], o[0]);
            split2<NPT>(-u0[2], -u0[3], o[1]);
            split2<NPT>(-u1[0], -u1[1], o[2]);
            split2<NPT>(-u1[2], -u1[3], o[3]);
#pragma unroll
            for (int m = 0; m < NPT; ++m) {
                const uint32_t r[4] = {o[0][m], o[1][m], o[2][m], o[3][m]};
                stsm4t(sX + m * kTriBytes + tri_block(i, warp) +
                           tri_piece((lane & 7) + (lane >> 4) * 8, lane >> 3 & 1),
                       r);
            }
            __syncwarp();
        }
        for (int i = warp; i < 4; ++i)
            leave(p.Tp, sh, NPT, i, warp, dsm + Lay::oT + tri_block(i, warp), kTriBytes);
    }
}

}  // namespace ss2d
