// ss2d_norm.cuh -- the block norms: the norm behind a mixer with its SiLU
// gate, the scaled residual sum, and the norm in front of the next block, in
// one pass over the rows, forward and backward.
//
// Per row of D values (float32 arithmetic; any part may be missing):
//     n  = (x - m) / sqrt(var + eps)   (layer)   or  x / sqrt(mean(x^2) + eps)  (rms)
//     t  = (n w_post + b_post) * SiLU(z)
//     r' = r + s t
//     n' = the norm of r',   y = n' w_pre + b_pre
// Backward, for dr' (the gradient of r' from behind) and dy:
//     G  = dr' + N'(dy w_pre)          dr = G
//     dt = s G                          ds = sum over rows of G t
//     dp = dt SiLU(z)                   dz = dt p SiLU'(z)   (p = n w_post + b_post)
//     dx = N(dp w_post)
//   with N(d) = rstd (d - n mean(d n) - [layer] mean(d)), and the weights'
//   gradients sums over the rows.
//
// Layout.  A row belongs to a team of TPR threads (a power of two, 1..512)
// that hold E of its values each in registers, so that a row is read once
// and its statistics are exact two-pass sums: the mean first, then the sum of
// squares about it.  Rows of 64 16-bit values are 8 lanes of one 16-byte
// vector each, four rows to a warp; teams of more than a warp sum through
// shared memory.  Every kernel is bound by the bytes of its rows.
//
// The backward's column sums (weights, biases, scale) are kept in registers
// over all the rows that a team visits, summed over the CTA's teams in
// order, written as one partial per CTA and summed by a second kernel in
// order: the same bits on every call.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ss2d_kernels.cuh"

namespace ss2d {

enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
constexpr int kNormCols = 5;   // ds, dw_post, dw_pre, db_post, db_pre

struct NormParams {
    const void *x, *z, *r;   // r: the residual (forward), r' as the forward stored it (backward)
    const float *s, *w_post, *b_post, *w_pre, *b_pre;
    void *r_out, *y;                  // forward
    const void *dr_out, *dy;          // backward
    void *dx, *dz, *dr;
    float *part;                      // [kNormCols][gridDim.x][D] partial column sums
    int cols;                         // bit c: column sum c is wanted
    long long rows, xs, zs;           // row i of x starts at (i / group) * xs + (i % group) * D
    int group;
    int D, tpr, post, pre;
    float eps;
};

// Thread t of a team holds vectors t, t + TPR, ... of V values of a row; a
// vector is 16 bytes of 16-bit values (8: V = 4), one or two 16-byte pieces of
// float32, or (V = 1) one value.  Rows are loaded as stored and converted when they are used, so that
// the next row can be on its way at half the registers.
template <typename T, int V>
struct NormVec {
    static constexpr int bytes = V * (int)sizeof(T), n = V == 1 ? 1 : bytes / 4;
    typename std::conditional<V == 1, T, uint32_t>::type w[n];
    __device__ __forceinline__ void load(const T *row, int col)
    {
        if constexpr (V == 1) {
            w[0] = row[col];
        } else if constexpr (bytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(row + col);
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < n / 4; ++i) {
                const uint4 u = reinterpret_cast<const uint4 *>(row + col)[i];
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            if constexpr (V == 1)
                w[i] = T(0.f);
            else
                w[i] = 0;
        }
    }
    __device__ __forceinline__ void get(float *v) const
    {
        if constexpr (V == 1) {
            v[0] = to_f32(w[0]);
        } else {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                if constexpr (sizeof(T) == 4) {
                    v[i] = __uint_as_float(w[i]);
                } else {
                    v[2 * i] = half_bits_to_f32<T>(w[i] & 0xffffu);
                    v[2 * i + 1] = half_bits_to_f32<T>(w[i] >> 16);
                }
            }
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void norm_load(const T *row, int col, float *v)
{
    NormVec<T, V> r;
    r.load(row, col);
    r.get(v);
}
// a row's vectors, zero past its end and for rows past the last
template <typename T, int V, int E>
struct NormRow {
    NormVec<T, V> v[E / V];
    template <typename On, typename Col>
    __device__ __forceinline__ void load(const T *row, bool live, On on, Col col)
    {
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            v[i].zero();
            if (live && on(i))
                v[i].load(row, col(i));
        }
    }
    __device__ __forceinline__ void get(float (&f)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E / V; ++i)
            v[i].get(f + i * V);
    }
};
template <typename T>
__device__ __forceinline__ T norm_round(float v)
{
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
        return __float2bfloat16_rn(v);
    else if constexpr (std::is_same_v<T, __half>)
        return __float2half_rn(v);
    else
        return v;
}
template <typename T, int V>
__device__ __forceinline__ void norm_store(T *row, int col, const float *v)
{
    if constexpr (V == 1) {
        row[col] = norm_round<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(row + col + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
        __align__(16) T h[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            h[i] = norm_round<T>(v[i]);
        if constexpr (V == 8)
            *reinterpret_cast<uint4 *>(row + col) = *reinterpret_cast<const uint4 *>(h);
        else
            *reinterpret_cast<uint2 *>(row + col) = *reinterpret_cast<const uint2 *>(h);
    }
}

// first value of row i of a tensor whose groups of rows are `gs` values apart
__device__ __forceinline__ long long norm_row(long long i, int group, long long gs, int D)
{
    if (group == 1)
        return i * gs;
    if (i >> 31)
        return i / group * gs + i % group * D;
    const unsigned o = (unsigned)i / (unsigned)group;
    return o * gs + (long long)((unsigned)i - o * (unsigned)group) * D;
}

// 1 / (1 + e^-z) on the multi-function unit: e^-z off by 2^-22 + 2^-23 |z|, the reciprocal by 2^-23 (relative);
// e^-z = inf gives 0
__device__ __forceinline__ float norm_sigmoid(float z) { return __fdividef(1.f, 1.f + mufu_ex2(-z * kLog2e)); }

// Sums over a team.  Teams up to a warp: butterfly shuffles inside the team
// (every lane ends with the same bits).  Larger teams: one value per warp
// through shared memory, added in warp order; two buffers in turn, so that
// one barrier per sum is enough (a buffer is rewritten two barriers later).
struct TeamSum {
    float2 *red;   // [2][32]
    int tpr, warp, w0, nw, buf;
    __device__ __forceinline__ void init(float2 *smem, int tpr_)
    {
        red = smem;
        tpr = tpr_;
        warp = threadIdx.x >> 5;
        nw = tpr >> 5;
        w0 = nw > 1 ? warp / nw * nw : 0;
        buf = 0;
    }
    // both sums at once
    __device__ __forceinline__ float2 operator()(float a, float b)
    {
        for (int o = (tpr < 32 ? tpr : 32) >> 1; o; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (nw > 1) {   // uniform over the CTA
            if ((threadIdx.x & 31) == 0)
                red[buf * 32 + warp] = make_float2(a, b);
            __syncthreads();
            a = b = 0.f;
            for (int i = 0; i < nw; ++i) {
                const float2 v = red[buf * 32 + w0 + i];
                a += v.x;
                b += v.y;
            }
            buf ^= 1;
        }
        return make_float2(a, b);
    }
    __device__ __forceinline__ float operator()(float a)
    {
        for (int o = (tpr < 32 ? tpr : 32) >> 1; o; o >>= 1)
            a += __shfl_xor_sync(0xffffffffu, a, o);
        if (nw > 1) {
            if ((threadIdx.x & 31) == 0)
                red[buf * 32 + warp].x = a;
            __syncthreads();
            a = 0.f;
            for (int i = 0; i < nw; ++i)
                a += red[buf * 32 + w0 + i].x;
            buf ^= 1;
        }
        return a;
    }
};

// v <- normalised v (values past the row's end stay zero); returns 1 / sqrt(. + eps)
template <int E, typename In>
__device__ __forceinline__ float norm_rows(float (&v)[E], int how, int D, float eps, TeamSum &sum, In in)
{
    const float invD = 1.f / (float)D;
    if (how == kNormLayer) {
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            a += v[e];
        const float m = sum(a) * invD;
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = in(e) ? v[e] - m : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        q = fmaf(v[e], v[e], q);
    const float rs = 1.f / sqrtf(sum(q) * invD + eps);
#pragma unroll
    for (int e = 0; e < E; ++e)
        v[e] *= rs;
    return rs;
}
// mean and 1 / sqrt(. + eps) of two rows at once (how none: 0 and 1), each as norm_rows has them
template <int E, typename GetA, typename GetB, typename In>
__device__ __forceinline__ void norm_stats2(GetA getA, int howA, GetB getB, int howB, int D, float eps, TeamSum &sum,
                                            In in, float2 &mean, float2 &rs)
{
    const float invD = 1.f / (float)D;
    mean = make_float2(0.f, 0.f);
    rs = make_float2(1.f, 1.f);
    float v[E];
    if (howA == kNormLayer || howB == kNormLayer) {
        float a = 0.f, b = 0.f;
        if (howA == kNormLayer) {
            getA(v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                a += v[e];
        }
        if (howB == kNormLayer) {
            getB(v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                b += v[e];
        }
        mean = sum(a, b);
        mean.x *= invD;
        mean.y *= invD;
    }
    if (howA == kNormNone && howB == kNormNone)
        return;
    float a = 0.f, b = 0.f;
    if (howA != kNormNone) {
        getA(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = in(e) ? v[e] - mean.x : 0.f;
            a = fmaf(d, d, a);
        }
    }
    if (howB != kNormNone) {
        getB(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = in(e) ? v[e] - mean.y : 0.f;
            b = fmaf(d, d, b);
        }
    }
    const float2 q = sum(a, b);
    if (howA != kNormNone)
        rs.x = 1.f / sqrtf(q.x * invD + eps);
    if (howB != kNormNone)
        rs.y = 1.f / sqrtf(q.y * invD + eps);
}
// d <- rs (d - n mean(d n) - [layer] mean(d))
template <int E, typename In>
__device__ __forceinline__ void norm_grad(float (&d)[E], const float (&n)[E], float rs, int how, int D,
                                          TeamSum &sum, In in)
{
    const float invD = 1.f / (float)D;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        a = fmaf(d[e], n[e], a);
        b += d[e];
    }
    float ma, mb = 0.f;
    if (how == kNormLayer) {
        const float2 m = sum(a, b);
        ma = m.x * invD;
        mb = m.y * invD;
    } else {
        ma = sum(a) * invD;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        d[e] = in(e) ? rs * (d[e] - n[e] * ma - mb) : 0.f;
}

// What a call has, as kernels are compiled for: the parts below, for rows that fill
// their teams (D = TPR * E), or kNormAny: whatever the parameters say.  With every part
// looked up and every column compared in the loop, the gated norm of 302592 rows of 64
// values issued 35 instructions a value and took 29 us, at 72 % of the issue slots.
enum { kHasPost = 1, kHasGate = 2, kHasRes = 4, kHasPre = 8, kHasScale = 16, kHasBias = 32, kNormAny = -1 };

// grid: CTAs of blockDim.x / tpr teams, one row per team and step; the next
// row's vectors are loaded as soon as this row's are converted, and a compiled
// combination keeps its weights in registers.
template <typename Tin, typename Tr, int V, int E, int M>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p)
{
    __shared__ float2 red[64];
    constexpr bool any = M == kNormAny;
    const bool post = any ? p.post != kNormNone : M & kHasPost, gate = any ? p.z != nullptr : M & kHasGate,
               res = any ? p.r != nullptr : M & kHasRes, pre = any ? p.pre != kNormNone : M & kHasPre,
               scale = any ? p.s != nullptr : M & kHasScale, bias = any || (M & kHasBias);
    const int lane = threadIdx.x % p.tpr, team = threadIdx.x / p.tpr, teams = blockDim.x / p.tpr;
    const int D = p.D;
    auto col = [&](int i) { return (lane + i * p.tpr) * V; };   // first column of vector i
    auto on = [&](int i) { return !any || col(i) < D; };
    auto in = [&](int e) { return !any || (lane + e / V * p.tpr) * V + e % V < D; };
    TeamSum sum;
    sum.init(red, p.tpr);
    // f(w, i): weights of vector i, from registers in a compiled combination
    constexpr int K = any ? 1 : E;
    float wq[K], wp[K], ws[K];
    auto keep = [&](const float *src, bool has, float (&w)[K]) {
        if constexpr (!any) {
            if (has) {
#pragma unroll
                for (int i = 0; i < E / V; ++i) {
                    if (src) {
                        norm_load<float, V>(src, col(i), w + i * V);
                    } else {
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            w[i * V + j] = 1.f;
                    }
                }
            }
        }
    };
    keep(p.w_post, post, wq);
    keep(p.w_pre, pre, wp);
    keep(p.s, scale, ws);
    auto times = [&](float *v, int i, const float *src, const float (&w)[K]) {
        if constexpr (!any) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] *= w[i * V + j];
        } else if (src) {
            float t[V];
            norm_load<float, V>(src, col(i), t);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] *= t[j];
        }
    };
    auto plus = [&](float *v, int i, const float *src) {
        if (bias && src) {
            float t[V];
            norm_load<float, V>(src, col(i), t);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] += t[j];
        }
    };
    const long long step = (long long)gridDim.x * teams;
    NormRow<Tin, V, E> xr, zr;
    NormRow<Tr, V, E> rr;
    auto load_x = [&](long long o) {
        const bool live = o < p.rows;
        xr.load(static_cast<const Tin *>(p.x) + (live ? norm_row(o, p.group, p.xs, D) : 0), live, on, col);
    };
    auto load_z = [&](long long o) {
        const bool live = o < p.rows;
        if (gate)
            zr.load(static_cast<const Tin *>(p.z) + (live ? norm_row(o, p.group, p.zs, D) : 0), live, on, col);
    };
    auto load_r = [&](long long o) {
        const bool live = o < p.rows;
        if (res)
            rr.load(static_cast<const Tr *>(p.r) + (live ? o * D : 0), live, on, col);
    };
    const long long first = (long long)blockIdx.x * teams;
    load_x(first + team);
    load_z(first + team);
    load_r(first + team);
    for (long long base = first; base < p.rows; base += step) {
        const long long o = base + team;
        const bool live = o < p.rows;
        float v[E], w[E];
        xr.get(v);
        load_x(o + step);
        if (post) {
            norm_rows<E>(v, p.post, D, p.eps, sum, in);
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (on(i)) {
                    times(v + i * V, i, p.w_post, wq);
                    plus(v + i * V, i, p.b_post);
                }
        }
        if (gate) {
            zr.get(w);
            load_z(o + step);
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] *= w[e] * norm_sigmoid(w[e]);
        }
        if (scale) {
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (on(i))
                    times(v + i * V, i, p.s, ws);
        }
        if (res) {
            rr.get(w);
            load_r(o + step);
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] += w[e];
        }
#pragma unroll
        for (int i = 0; i < E / V; ++i)
            if (live && on(i))
                norm_store<Tr, V>(static_cast<Tr *>(p.r_out) + o * D, col(i), v + i * V);
        if (pre) {
            // the norm reads r' before its rounding to r's type
            norm_rows<E>(v, p.pre, D, p.eps, sum, in);
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (on(i)) {
                    times(v + i * V, i, p.w_pre, wp);
                    plus(v + i * V, i, p.b_pre);
                    if (live)
                        norm_store<Tin, V>(static_cast<Tin *>(p.y) + o * D, col(i), v + i * V);
                }
        }
    }
}

// dynamic shared memory: blockDim.x * E floats (the teams' column sums).  BIAS:
// the sums for biases are kept too (two of five, 16 registers).  The next row's
// vectors are on their way while a row's sums go round, and both norms' statistics
// go round together: with loads where they are used and every sum by itself,
// 12544 rows of 1024 values with every part took 144 us.
template <typename Tin, typename Tr, int V, int E, bool BIAS, int M>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p)
{
    constexpr int NC = BIAS ? kNormCols : 3;
    constexpr bool ahead = E < 16;   // rows of 4097 values and more have no registers for it
    extern __shared__ __align__(16) float csum[];
    __shared__ float2 red[64];
    const int lane = threadIdx.x % p.tpr, team = threadIdx.x / p.tpr, teams = blockDim.x / p.tpr;
    constexpr bool any = M == kNormAny;
    const bool post = any ? p.post != kNormNone : M & kHasPost, gate = any ? p.z != nullptr : M & kHasGate,
               pre = any ? p.pre != kNormNone : M & kHasPre, scale = any ? p.s != nullptr : M & kHasScale,
               bias = any || (M & kHasBias);
    const int D = p.D;
    auto col = [&](int i) { return (lane + i * p.tpr) * V; };
    auto on = [&](int i) { return !any || col(i) < D; };
    auto in = [&](int e) { return !any || (lane + e / V * p.tpr) * V + e % V < D; };
    TeamSum sum;
    sum.init(red, p.tpr);
    float acc[NC][E];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[c][e] = 0.f;
    auto vec = [&](const float *w, int i, float one, float (&o)[V]) {
        if (w) {
            norm_load<float, V>(w, col(i), o);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                o[j] = one;
        }
    };
    const long long step = (long long)gridDim.x * teams;
    NormRow<Tin, V, E> xr, zr, yr;
    NormRow<Tr, V, E> rr, gr;
    auto row_x = [&](long long o) {
        const bool live = o < p.rows;
        xr.load(static_cast<const Tin *>(p.x) + (live ? norm_row(o, p.group, p.xs, D) : 0), live, on, col);
    };
    auto row_z = [&](long long o) {
        const bool live = o < p.rows;
        if (gate)
            zr.load(static_cast<const Tin *>(p.z) + (live ? norm_row(o, p.group, p.zs, D) : 0), live, on, col);
    };
    auto row_pre = [&](long long o) {
        const bool live = o < p.rows;
        if (pre) {
            rr.load(static_cast<const Tr *>(p.r) + (live ? o * D : 0), live, on, col);
            yr.load(static_cast<const Tin *>(p.dy) + (live ? o * D : 0), live, on, col);
        }
    };
    auto row_g = [&](long long o) {
        const bool live = o < p.rows;
        if (p.dr_out)
            gr.load(static_cast<const Tr *>(p.dr_out) + (live ? o * D : 0), live, on, col);
    };
    const long long first = (long long)blockIdx.x * teams;
    if constexpr (ahead) {
        row_pre(first + team);
        row_g(first + team);
        row_x(first + team);
        row_z(first + team);
    }
    for (long long base = first; base < p.rows; base += step) {
        const long long o = base + team;
        const bool live = o < p.rows;
        float g[E], a[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            g[e] = 0.f;
        if constexpr (!ahead) {
            row_pre(o);
            row_g(o);
            row_x(o);
            row_z(o);
        }
        // both norms' statistics in one round of sums
        float2 mean, rs;
        norm_stats2<E>([&](float (&v)[E]) { rr.get(v); }, pre ? p.pre : kNormNone,
                       [&](float (&v)[E]) { xr.get(v); }, post ? p.post : kNormNone, D, p.eps,
                       sum, in, mean, rs);
        // G: the gradient of r'
        if (pre) {
            rr.get(a);
            yr.get(g);
            if constexpr (ahead)
                row_pre(o + step);
#pragma unroll
            for (int e = 0; e < E; ++e)
                a[e] = in(e) ? (a[e] - mean.x) * rs.x : 0.f;
#pragma unroll
            for (int i = 0; i < E / V; ++i) {
                float w[V];
                if (on(i))
                    vec(p.w_pre, i, 1.f, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = i * V + j;
                    acc[2][e] = fmaf(g[e], a[e], acc[2][e]);
                    if constexpr (BIAS)
                        acc[4][e] += g[e];
                    g[e] = on(i) ? g[e] * w[j] : 0.f;
                }
            }
            norm_grad<E>(g, a, rs.x, p.pre, D, sum, in);
        }
        if (p.dr_out) {
            gr.get(a);
            if constexpr (ahead)
                row_g(o + step);
#pragma unroll
            for (int e = 0; e < E; ++e)
                g[e] += a[e];
        }
        if (p.dr) {
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (live && on(i))
                    norm_store<Tr, V>(static_cast<Tr *>(p.dr) + o * D, col(i), g + i * V);
        }
        // the branch again: n, p, t
        xr.get(a);
        if constexpr (ahead)
            row_x(o + step);
        if (post) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                a[e] = in(e) ? (a[e] - mean.y) * rs.y : 0.f;
        }
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            float w[V], b[V], s[V], z[V], dz[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                w[j] = b[j] = s[j] = z[j] = 0.f;
            if (on(i)) {
                vec(post ? p.w_post : nullptr, i, 1.f, w);
                vec(post && bias ? p.b_post : nullptr, i, 0.f, b);
                vec(scale ? p.s : nullptr, i, 1.f, s);
            }
            if (gate)
                zr.v[i].get(z);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = i * V + j;
                const float pv = fmaf(a[e], w[j], b[j]);
                float gt = 1.f, dgate = 0.f;
                if (gate) {
                    const float sg = norm_sigmoid(z[j]);
                    gt = z[j] * sg;
                    dgate = sg * fmaf(z[j], 1.f - sg, 1.f);
                }
                if (scale)
                    acc[0][e] = fmaf(g[e], pv * gt, acc[0][e]);
                const float dt = s[j] * g[e];
                dz[j] = dt * pv * dgate;
                const float dp = dt * gt;
                acc[1][e] = fmaf(dp, a[e], acc[1][e]);
                if constexpr (BIAS)
                    acc[3][e] += dp;
                g[e] = dp * w[j];
            }
            if (gate && p.dz && live && on(i))
                norm_store<Tin, V>(static_cast<Tin *>(p.dz) + o * D, col(i), dz);
        }
        if constexpr (ahead)
            row_z(o + step);
        if (post)
            norm_grad<E>(g, a, rs.y, p.post, D, sum, in);
#pragma unroll
        for (int i = 0; i < E / V; ++i)
            if (live && on(i))
                norm_store<Tin, V>(static_cast<Tin *>(p.dx) + o * D, col(i), g + i * V);
    }
    // the CTA's column sums, its teams in order
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (!(p.cols >> c & 1))
            continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e)
            csum[(team * E + e) * p.tpr + lane] = acc[c][e];
        __syncthreads();
        for (int i = threadIdx.x; i < p.tpr * E; i += blockDim.x) {
            const int e = i / p.tpr, l = i % p.tpr;
            const int d = (l + e / V * p.tpr) * V + e % V;
            if (d >= D)
                continue;
            float v = 0.f;
            for (int t = 0; t < teams; ++t)
                v += csum[(t * E + e) * p.tpr + l];
            p.part[((size_t)c * gridDim.x + blockIdx.x) * D + d] = v;
        }
    }
}

struct NormSums {
    float *out[kNormCols];
};
// out[c][d] = sum over the partials, in order: 32 interleaved runs of CTAs, then the runs.  grid (ceil(D / 32),
// kNormCols), 1024 threads (256 threads and 8 runs took 15 us for 296 partials of 1024 columns)
static __global__ void __launch_bounds__(1024) norm_colsum_kernel(const float *part, NormSums o, int nparts, int D)
{
    __shared__ float sm[32][33];
    float *out = o.out[blockIdx.y];
    if (!out)
        return;
    const int lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane, run = threadIdx.x >> 5;
    float v = 0.f;
    if (d < D) {
#pragma unroll 4
        for (int i = run; i < nparts; i += 32)
            v += part[((size_t)blockIdx.y * nparts + i) * D + d];
    }
    sm[run][lane] = v;
    __syncthreads();
    // warp `run` sums column `run`
    v = sm[lane][run];
    for (int m = 16; m; m >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    if (lane == 0 && blockIdx.x * 32 + run < D)
        out[blockIdx.x * 32 + run] = v;
}

}  // namespace ss2d
