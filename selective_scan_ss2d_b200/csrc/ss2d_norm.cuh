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
constexpr int kNormCols = 5;   // ds, dw_post, db_post, dw_pre, db_pre

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

// E values of one row: thread t of a team holds vectors t, t + TPR, ... of V values
template <typename T, int V>
__device__ __forceinline__ void norm_load(const T *row, int col, float *v)
{
    if constexpr (V == 1) {
        v[0] = to_f32(row[col]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(row + col + i);
            v[i] = f.x;
            v[i + 1] = f.y;
            v[i + 2] = f.z;
            v[i + 3] = f.w;
        }
    } else {
        static_assert(V % 8 == 0, "16-byte vectors");
        const uint4 u = *reinterpret_cast<const uint4 *>(row + col);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = half_bits_to_f32<T>(w[i] & 0xffffu);
            v[2 * i + 1] = half_bits_to_f32<T>(w[i] >> 16);
        }
    }
}
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
        __align__(16) T h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = norm_round<T>(v[i]);
        *reinterpret_cast<uint4 *>(row + col) = *reinterpret_cast<const uint4 *>(h);
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

// Sums over a team.  Teams up to a warp: butterfly shuffles inside the team
// (every lane ends with the same bits).  Larger teams: one value per warp
// through shared memory, added in warp order; two buffers in turn, so that
// one barrier per sum is enough (a buffer is rewritten two barriers later).
struct TeamSum {
    float *red;   // [2][32]
    int tpr, warp, w0, nw, buf;
    __device__ __forceinline__ void init(float *smem, int tpr_)
    {
        red = smem;
        tpr = tpr_;
        warp = threadIdx.x >> 5;
        nw = tpr >> 5;
        w0 = nw > 1 ? warp / nw * nw : 0;
        buf = 0;
    }
    __device__ __forceinline__ float operator()(float v)
    {
        for (int o = (tpr < 32 ? tpr : 32) >> 1; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if (nw > 1) {   // uniform over the CTA
            if ((threadIdx.x & 31) == 0)
                red[buf * 32 + warp] = v;
            __syncthreads();
            v = 0.f;
            for (int i = 0; i < nw; ++i)
                v += red[buf * 32 + w0 + i];
            buf ^= 1;
        }
        return v;
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
    const float ma = sum(a) * invD;
    const float mb = how == kNormLayer ? sum(b) * invD : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        d[e] = in(e) ? rs * (d[e] - n[e] * ma - mb) : 0.f;
}

// grid: CTAs of blockDim.x / tpr teams, one row per team and step
template <typename Tin, typename Tr, int V, int E>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p)
{
    __shared__ float red[64];
    const int lane = threadIdx.x % p.tpr, team = threadIdx.x / p.tpr, teams = blockDim.x / p.tpr;
    const int D = p.D;
    auto col = [&](int i) { return (lane + i * p.tpr) * V; };   // first column of vector i
    auto in = [&](int e) { return (lane + e / V * p.tpr) * V + e % V < D; };
    TeamSum sum;
    sum.init(red, p.tpr);
    const long long step = (long long)gridDim.x * teams;
    for (long long base = (long long)blockIdx.x * teams; base < p.rows; base += step) {
        const long long row = base + team;
        const bool live = row < p.rows;
        const long long o = live ? row : 0;
        const Tin *xr = static_cast<const Tin *>(p.x) + norm_row(o, p.group, p.xs, D);
        const Tin *zr = static_cast<const Tin *>(p.z) + norm_row(o, p.group, p.zs, D);
        const Tr *rr = static_cast<const Tr *>(p.r) + o * D;
        float v[E], z[E], r[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = z[e] = r[e] = 0.f;
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            if (live && col(i) < D) {
                norm_load<Tin, V>(xr, col(i), v + i * V);
                if (p.z)
                    norm_load<Tin, V>(zr, col(i), z + i * V);
                if (p.r)
                    norm_load<Tr, V>(rr, col(i), r + i * V);
            }
        }
        if (p.post != kNormNone) {
            norm_rows<E>(v, p.post, D, p.eps, sum, in);
#pragma unroll
            for (int i = 0; i < E / V; ++i) {
                if (col(i) >= D)
                    continue;
                float w[V];
                if (p.w_post) {
                    norm_load<float, V>(p.w_post, col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        v[i * V + j] *= w[j];
                }
                if (p.b_post) {
                    norm_load<float, V>(p.b_post, col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        v[i * V + j] += w[j];
                }
            }
        }
        if (p.z) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] *= z[e] / (1.f + expf(-z[e]));
        }
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            if (col(i) >= D)
                continue;
            if (p.s) {
                float w[V];
                norm_load<float, V>(p.s, col(i), w);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[i * V + j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[i * V + j] += r[i * V + j];
            if (live)
                norm_store<Tr, V>(static_cast<Tr *>(p.r_out) + o * D, col(i), v + i * V);
        }
        if (p.pre != kNormNone) {
            // the norm reads r' before its rounding to r's type
            norm_rows<E>(v, p.pre, D, p.eps, sum, in);
#pragma unroll
            for (int i = 0; i < E / V; ++i) {
                if (col(i) >= D)
                    continue;
                float w[V];
                if (p.w_pre) {
                    norm_load<float, V>(p.w_pre, col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        v[i * V + j] *= w[j];
                }
                if (p.b_pre) {
                    norm_load<float, V>(p.b_pre, col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        v[i * V + j] += w[j];
                }
                if (live)
                    norm_store<Tin, V>(static_cast<Tin *>(p.y) + o * D, col(i), v + i * V);
            }
        }
    }
}

// dynamic shared memory: blockDim.x * E floats (the teams' column sums)
template <typename Tin, typename Tr, int V, int E>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p)
{
    extern __shared__ __align__(16) float csum[];
    __shared__ float red[64];
    const int lane = threadIdx.x % p.tpr, team = threadIdx.x / p.tpr, teams = blockDim.x / p.tpr;
    const int D = p.D;
    auto col = [&](int i) { return (lane + i * p.tpr) * V; };
    auto in = [&](int e) { return (lane + e / V * p.tpr) * V + e % V < D; };
    TeamSum sum;
    sum.init(red, p.tpr);
    float acc[kNormCols][E];
#pragma unroll
    for (int c = 0; c < kNormCols; ++c)
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
    for (long long base = (long long)blockIdx.x * teams; base < p.rows; base += step) {
        const long long row = base + team;
        const bool live = row < p.rows;
        const long long o = live ? row : 0;
        float g[E], a[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            g[e] = a[e] = 0.f;
        // G: the gradient of r'
        if (p.pre != kNormNone) {
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (live && col(i) < D) {
                    norm_load<Tr, V>(static_cast<const Tr *>(p.r) + o * D, col(i), a + i * V);
                    norm_load<Tin, V>(static_cast<const Tin *>(p.dy) + o * D, col(i), g + i * V);
                }
            const float rs = norm_rows<E>(a, p.pre, D, p.eps, sum, in);
#pragma unroll
            for (int i = 0; i < E / V; ++i) {
                float w[V];
                if (col(i) < D)
                    vec(p.w_pre, i, 1.f, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = i * V + j;
                    acc[3][e] = fmaf(g[e], a[e], acc[3][e]);
                    acc[4][e] += g[e];
                    g[e] = col(i) < D ? g[e] * w[j] : 0.f;
                }
            }
            norm_grad<E>(g, a, rs, p.pre, D, sum, in);
        }
        if (p.dr_out) {
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (live && col(i) < D) {
                    float w[V];
                    norm_load<Tr, V>(static_cast<const Tr *>(p.dr_out) + o * D, col(i), w);
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        g[i * V + j] += w[j];
                }
        }
        if (p.dr) {
#pragma unroll
            for (int i = 0; i < E / V; ++i)
                if (live && col(i) < D)
                    norm_store<Tr, V>(static_cast<Tr *>(p.dr) + o * D, col(i), g + i * V);
        }
        // the branch again: n, p, t
        const Tin *xr = static_cast<const Tin *>(p.x) + norm_row(o, p.group, p.xs, D);
#pragma unroll
        for (int e = 0; e < E; ++e)
            a[e] = 0.f;
#pragma unroll
        for (int i = 0; i < E / V; ++i)
            if (live && col(i) < D)
                norm_load<Tin, V>(xr, col(i), a + i * V);
        float rs = 0.f;
        if (p.post != kNormNone)
            rs = norm_rows<E>(a, p.post, D, p.eps, sum, in);
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            const bool on = live && col(i) < D;
            float w[V], b[V], s[V], z[V], dz[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                w[j] = b[j] = s[j] = z[j] = 0.f;
            if (col(i) < D) {
                vec(p.post != kNormNone ? p.w_post : nullptr, i, 1.f, w);
                vec(p.post != kNormNone ? p.b_post : nullptr, i, 0.f, b);
                vec(p.s, i, 1.f, s);
            }
            if (p.z && on)
                norm_load<Tin, V>(static_cast<const Tin *>(p.z) + norm_row(o, p.group, p.zs, D), col(i), z);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int e = i * V + j;
                const float pv = fmaf(a[e], w[j], b[j]);
                float gate = 1.f, dgate = 0.f;
                if (p.z) {
                    const float sg = 1.f / (1.f + expf(-z[j]));
                    gate = z[j] * sg;
                    dgate = sg * fmaf(z[j], 1.f - sg, 1.f);
                }
                acc[0][e] = fmaf(g[e], pv * gate, acc[0][e]);
                const float dt = s[j] * g[e];
                dz[j] = dt * pv * dgate;
                const float dp = dt * gate;
                acc[1][e] = fmaf(dp, a[e], acc[1][e]);
                acc[2][e] += dp;
                g[e] = dp * w[j];
            }
            if (p.dz && on)
                norm_store<Tin, V>(static_cast<Tin *>(p.dz) + o * D, col(i), dz);
        }
        if (p.post != kNormNone)
            norm_grad<E>(g, a, rs, p.post, D, sum, in);
#pragma unroll
        for (int i = 0; i < E / V; ++i)
            if (live && col(i) < D)
                norm_store<Tin, V>(static_cast<Tin *>(p.dx) + o * D, col(i), g + i * V);
    }
    // the CTA's column sums, its teams in order
#pragma unroll
    for (int c = 0; c < kNormCols; ++c) {
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
// out[c][d] = sum over the partials, in order: 8 interleaved runs of CTAs, then the runs.  grid (ceil(D / 32),
// kNormCols), 256 threads
static __global__ void __launch_bounds__(256) norm_colsum_kernel(const float *part, NormSums o, int nparts, int D)
{
    __shared__ float sm[8][32];
    float *out = o.out[blockIdx.y];
    if (!out)
        return;
    const int d = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
    float v = 0.f;
    if (d < D)
        for (int i = run; i < nparts; i += 8)
            v += part[((size_t)blockIdx.y * nparts + i) * D + d];
    sm[run][threadIdx.x & 31] = v;
    __syncthreads();
    if (run == 0 && d < D) {
        v = sm[0][threadIdx.x];
        for (int i = 1; i < 8; ++i)
            v += sm[i][threadIdx.x];
        out[d] = v;
    }
}

}  // namespace ss2d
