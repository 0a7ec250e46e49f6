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
// shared memory.  What bounds a form is said at its kernel: the bytes of its rows
// in the gated head norm, which runs at four fifths of the copy rate, before
// them two waves of CTAs in wider forward rows, and the rounds of sums in the backward.
//
// The backward's column sums (weights, biases, scale) are kept in registers
// over all the rows that a team visits and summed over the CTA's teams in
// order.  The CTAs' sums are partials that a second kernel adds up in order or,
// for few rows, stay in the shared memory of one cluster, which adds them up
// itself: the same bits on every call either way.
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
    float *part;                      // [kNormCols][gridDim.x][D] partial column sums (null: the grid is one cluster)
    float *sums[kNormCols];           // column sums that a cluster writes itself
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
        uint32_t h[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same_v<T, __half>) {
                const __half2 t = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                h[i] = *reinterpret_cast<const uint32_t *>(&t);
            } else {
                const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                h[i] = *reinterpret_cast<const uint32_t *>(&t);
            }
        }
        if constexpr (V == 8)
            *reinterpret_cast<uint4 *>(row + col) = make_uint4(h[0], h[1], h[2], h[3]);
        else
            *reinterpret_cast<uint2 *>(row + col) = make_uint2(h[0], h[1]);
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
__device__ __forceinline__ float norm_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 norm_sigmoid2(float2 z)
{
    const float2 t = __fmul2_rn(z, make_float2(-kLog2e, -kLog2e));
    const float2 e = __fadd2_rn(make_float2(mufu_ex2(t.x), mufu_ex2(t.y)), make_float2(1.f, 1.f));
    return make_float2(norm_rcp(e.x), norm_rcp(e.y));
}

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
        if (tpr >= 32) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
        } else {
            for (int o = tpr >> 1; o; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
        }
        if (nw > 1) {   // uniform over the CTA
            float2 *r = red + buf * 32;
            if ((threadIdx.x & 31) == 0)
                r[warp] = make_float2(a, b);
            __syncthreads();
            a = b = 0.f;
            for (int i = 0; i < nw; i += 2) {   // two warps' sums to a read
                const float4 v = *reinterpret_cast<const float4 *>(r + w0 + i);
                a += v.x + v.z;
                b += v.y + v.w;
            }
            buf ^= 1;
        }
        return make_float2(a, b);
    }
    __device__ __forceinline__ float operator()(float a)
    {
        if (tpr >= 32) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                a += __shfl_xor_sync(0xffffffffu, a, o);
        } else {
            for (int o = tpr >> 1; o; o >>= 1)
                a += __shfl_xor_sync(0xffffffffu, a, o);
        }
        if (nw > 1) {
            float *r = reinterpret_cast<float *>(red + buf * 32);
            if ((threadIdx.x & 31) == 0)
                r[warp] = a;
            __syncthreads();
            a = 0.f;
            for (int i = 0; i < nw; i += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(r + w0 + i);
                a += v.x + v.y;
            }
            buf ^= 1;
        }
        return a;
    }
};

// Pairs of a thread's values, on the packed float32 instructions (each lane
// rounds as the single one does): the kernels are bound by instructions before bytes.
__device__ __forceinline__ float2 pair(const float *v, int k) { return make_float2(v[2 * k], v[2 * k + 1]); }
__device__ __forceinline__ void set_pair(float *v, int k, float2 x)
{
    v[2 * k] = x.x;
    v[2 * k + 1] = x.y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <int E>
__device__ __forceinline__ float norm_total(const float (&v)[E])
{
    float2 a = pair(v, 0);
#pragma unroll
    for (int k = 1; k < E / 2; ++k)
        a = __fadd2_rn(a, pair(v, k));
    return a.x + a.y;
}
template <int E>
__device__ __forceinline__ float norm_dot(const float (&v)[E], const float (&w)[E])
{
    float2 a = __fmul2_rn(pair(v, 0), pair(w, 0));
#pragma unroll
    for (int k = 1; k < E / 2; ++k)
        a = __ffma2_rn(pair(v, k), pair(w, k), a);
    return a.x + a.y;
}
// v <- v - m, values past the row's end stay zero
template <int E, typename In>
__device__ __forceinline__ void norm_shift(float (&v)[E], float m, In in)
{
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        const float2 d = __fadd2_rn(pair(v, k), both(-m));
        v[2 * k] = in(2 * k) ? d.x : 0.f;
        v[2 * k + 1] = in(2 * k + 1) ? d.y : 0.f;
    }
}
template <int E>
__device__ __forceinline__ void norm_times(float (&v)[E], float f)
{
#pragma unroll
    for (int k = 0; k < E / 2; ++k)
        set_pair(v, k, __fmul2_rn(pair(v, k), both(f)));
}

// v <- normalised v (values past the row's end stay zero)
template <int E, typename In>
__device__ __forceinline__ void norm_rows(float (&v)[E], int how, int D, float eps, TeamSum &sum, In in)
{
    const float invD = 1.f / (float)D;
    if (how == kNormLayer)
        norm_shift<E>(v, sum(norm_total<E>(v)) * invD, in);
    norm_times<E>(v, rsqrtf(sum(norm_dot<E>(v, v)) * invD + eps));
}
// mean and 1 / sqrt(. + eps) of two rows at once (how none: 0 and 1), each as norm_rows has them
template <int E, typename GetA, typename GetB, typename In>
__device__ __forceinline__ void norm_stats2(GetA getA, int howA, GetB getB, int howB, int D, float eps, TeamSum &sum,
                                            In in, float2 &mean, float2 &rs)
{
    const float invD = 1.f / (float)D;
    mean = make_float2(0.f, 0.f);
    rs = make_float2(1.f, 1.f);
    if (howA == kNormNone && howB == kNormNone)
        return;
    float v[E], a = 0.f, b = 0.f;
    if (howA == kNormLayer || howB == kNormLayer) {
        if (howA == kNormLayer) {
            getA(v);
            a = norm_total<E>(v);
        }
        if (howB == kNormLayer) {
            getB(v);
            b = norm_total<E>(v);
        }
        mean = sum(a, b);
        mean.x *= invD;
        mean.y *= invD;
        a = b = 0.f;
    }
    if (howA != kNormNone) {
        getA(v);
        if (howA == kNormLayer)
            norm_shift<E>(v, mean.x, in);
        a = norm_dot<E>(v, v);
    }
    if (howB != kNormNone) {
        getB(v);
        if (howB == kNormLayer)
            norm_shift<E>(v, mean.y, in);
        b = norm_dot<E>(v, v);
    }
    const float2 q = sum(a, b);
    if (howA != kNormNone)
        rs.x = rsqrtf(q.x * invD + eps);
    if (howB != kNormNone)
        rs.y = rsqrtf(q.y * invD + eps);
}
// d <- rs (d - n mean(d n) - [layer] mean(d))
template <int E, typename In>
__device__ __forceinline__ void norm_grad(float (&d)[E], const float (&n)[E], float rs, int how, int D,
                                          TeamSum &sum, In in)
{
    const float f = rs / (float)D, a = norm_dot<E>(d, n);
    float2 m = make_float2(0.f, 0.f);
    if (how == kNormLayer)
        m = sum(a, norm_total<E>(d));
    else
        m.x = sum(a);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        float2 t = __ffma2_rn(pair(n, k), both(-m.x * f), __fmul2_rn(pair(d, k), both(rs)));
        if (how == kNormLayer)
            t = __fadd2_rn(t, both(-m.y * f));
        d[2 * k] = in(2 * k) ? t.x : 0.f;
        d[2 * k + 1] = in(2 * k + 1) ? t.y : 0.f;
    }
}

// What a call has, as kernels are compiled for: the parts below, for rows that fill
// their teams (D = TPR * E), or kNormAny: whatever the parameters say.  With every part
// looked up and every column compared in the loop, the gated norm of 302592 rows of 64
// values issued 35 instructions a value and took 29 us, at 72 % of the issue slots; with
// the combination compiled and packed arithmetic 22 us.
enum { kHasPost = 1, kHasGate = 2, kHasRes = 4, kHasPre = 8, kHasScale = 16, kHasBias = 32, kNormAny = -1 };

// grid: CTAs of blockDim.x / tpr teams, one row per team and step; the next
// row's vectors are loaded as soon as this row's are converted, and a compiled
// combination keeps its weights in registers.
template <typename Tin, typename Tr, int V, int E, int M>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p)
{
    __shared__ __align__(16) float2 red[64];
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
            for (int k = 0; k < V / 2; ++k)
                set_pair(v, k, __fmul2_rn(pair(v, k), pair(w + i * V, k)));
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
            for (int k = 0; k < E / 2; ++k)
                set_pair(v, k, __fmul2_rn(pair(v, k), __fmul2_rn(pair(w, k), norm_sigmoid2(pair(w, k)))));
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
            for (int k = 0; k < E / 2; ++k)
                set_pair(v, k, __fadd2_rn(pair(v, k), pair(w, k)));
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

// Every CTA of the cluster is here, what they wrote to shared memory can be read; a float of CTA `rank`
__device__ __forceinline__ void norm_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");   // lanes may come apart
}
__device__ __forceinline__ float norm_cluster_read(const float *v, unsigned rank)
{
    float f;
    asm volatile("{\n.reg .u32 a;\nmapa.shared::cluster.u32 a, %1, %2;\nld.shared::cluster.f32 %0, [a];\n}"
                 : "=f"(f)
                 : "r"((unsigned)__cvta_generic_to_shared(v)), "r"(rank)
                 : "memory");
    return f;
}

// CTAs of 256 threads per SM of the compiled combinations
__host__ __device__ constexpr int norm_bwd_ctas(int E) { return E == 8 ? 3 : 2; }

// dynamic shared memory: blockDim.x * E floats (the teams' column sums).  BIAS:
// the sums for biases are kept too (two of five, 16 registers).  Both norms'
// statistics go round the team together.  Measured on 12544 rows of 1024 values with every
// part: loads where they are used and every sum by itself 144 us; the next row ahead 94;
// compiled combinations 69; packed arithmetic, unrolled sums and three CTAs 65 (2.6 TB/s,
// 63 % of the issue slots: the rounds of sums, a third of the instructions, bound it).
template <typename Tin, typename Tr, int V, int E, bool BIAS, int M>
__global__ void __launch_bounds__(M == kNormAny ? 512 : 256, M == kNormAny ? 1 : norm_bwd_ctas(E)) norm_bwd_kernel(const NormParams p)
{
    constexpr int NC = BIAS ? kNormCols : 3;
    // next row ahead, or a third CTA per SM, which hides as much; rows of 4097 values and more have registers for neither
    constexpr bool ahead = M == kNormAny ? E < 16 : norm_bwd_ctas(E) == 2;
    extern __shared__ __align__(16) float csum[];
    __shared__ __align__(16) float2 red[64];
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
    // a weight's values of the thread's columns, `one` where it is not there or past the row's end
    auto weights = [&](const float *w, float one, float (&o)[E]) {
#pragma unroll
        for (int i = 0; i < E / V; ++i) {
            if (w && on(i)) {
                norm_load<float, V>(w, col(i), o + i * V);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    o[i * V + j] = one;
            }
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
        // a team past the last row holds zeros: with eps = 0 its 1 / sqrt is infinite, and 0 * inf would go into the
        // column sums
        rs = live ? rs : make_float2(0.f, 0.f);
        // G: the gradient of r'
        if (pre) {
            rr.get(a);
            yr.get(g);
            if constexpr (ahead)
                row_pre(o + step);
            if (p.pre == kNormLayer)
                norm_shift<E>(a, mean.x, in);
            norm_times<E>(a, rs.x);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                const float2 gk = pair(g, k);
                set_pair(acc[2], k, __ffma2_rn(gk, pair(a, k), pair(acc[2], k)));
                if constexpr (BIAS)
                    set_pair(acc[4], k, __fadd2_rn(gk, pair(acc[4], k)));
            }
            float w[E];
            weights(p.w_pre, 1.f, w);
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                set_pair(g, k, __fmul2_rn(pair(g, k), pair(w, k)));
            norm_grad<E>(g, a, rs.x, p.pre, D, sum, in);
        }
        if (p.dr_out) {
            gr.get(a);
            if constexpr (ahead)
                row_g(o + step);
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                set_pair(g, k, __fadd2_rn(pair(g, k), pair(a, k)));
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
            if (p.post == kNormLayer)
                norm_shift<E>(a, mean.y, in);
            norm_times<E>(a, rs.y);
        }
        {
            float w[E], z[E];   // w_post, s
            weights(post ? p.w_post : nullptr, 1.f, w);
            weights(scale ? p.s : nullptr, 1.f, z);
            float pv[E];
            if (post && bias && p.b_post) {
                weights(p.b_post, 0.f, pv);
#pragma unroll
                for (int k = 0; k < E / 2; ++k)
                    set_pair(pv, k, __ffma2_rn(pair(a, k), pair(w, k), pair(pv, k)));
            } else {
#pragma unroll
                for (int k = 0; k < E / 2; ++k)
                    set_pair(pv, k, post ? __fmul2_rn(pair(a, k), pair(w, k)) : pair(a, k));
            }
            // g: G, then dt = s G; ds takes G t, t = p SiLU(z)
            if (gate) {
                float zz[E];
                zr.get(zz);
#pragma unroll
                for (int k = 0; k < E / 2; ++k) {
                    const float2 zk = pair(zz, k), sg = norm_sigmoid2(zk), gt = __fmul2_rn(zk, sg);
                    const float2 gk = pair(g, k), pk = pair(pv, k);
                    if (scale)
                        set_pair(acc[0], k, __ffma2_rn(gk, __fmul2_rn(pk, gt), pair(acc[0], k)));
                    const float2 dt = scale ? __fmul2_rn(gk, pair(z, k)) : gk;
                    // SiLU'(z) = sg (1 + z (1 - sg)) = sg + z sg - (z sg) sg
                    const float2 dg = __ffma2_rn(gt, __ffma2_rn(sg, both(-1.f), both(1.f)), sg);
                    set_pair(zz, k, __fmul2_rn(__fmul2_rn(dt, pk), dg));
                    set_pair(g, k, __fmul2_rn(dt, gt));   // dp
                }
                if (p.dz) {
#pragma unroll
                    for (int i = 0; i < E / V; ++i)
                        if (live && on(i))
                            norm_store<Tin, V>(static_cast<Tin *>(p.dz) + o * D, col(i), zz + i * V);
                }
            } else if (scale) {
#pragma unroll
                for (int k = 0; k < E / 2; ++k) {
                    const float2 gk = pair(g, k);
                    set_pair(acc[0], k, __ffma2_rn(gk, pair(pv, k), pair(acc[0], k)));
                    set_pair(g, k, __fmul2_rn(gk, pair(z, k)));
                }
            }
            if (post) {
#pragma unroll
                for (int k = 0; k < E / 2; ++k) {
                    const float2 dp = pair(g, k);
                    set_pair(acc[1], k, __ffma2_rn(dp, pair(a, k), pair(acc[1], k)));
                    if constexpr (BIAS)
                        set_pair(acc[3], k, __fadd2_rn(dp, pair(acc[3], k)));
                    set_pair(g, k, __fmul2_rn(dp, pair(w, k)));
                }
            }
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
    // the CTA's column sums, its teams in order; a cluster keeps them in shared memory behind csum
    float *mine = csum + blockDim.x * E;
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
            if (p.part)
                p.part[((size_t)c * gridDim.x + blockIdx.x) * D + d] = v;
            else
                mine[c * D + d] = v;
        }
    }
    if (p.cols && !p.part) {
        norm_cluster_sync();
        for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < NC * D; i += gridDim.x * blockDim.x) {
            const int c = i / D;
            if (!(p.cols >> c & 1))
                continue;
            float v = 0.f;
            for (unsigned r = 0; r < gridDim.x; ++r)
                v += norm_cluster_read(mine + i, r);
            p.sums[c][i - c * D] = v;
        }
        norm_cluster_sync();   // no CTA leaves while its sums are read
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
