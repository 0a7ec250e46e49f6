// ss2d_norm.cu -- the C ABI of the block norms (include/ss2d.h): argument
// checks, thread layout and launches.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "ss2d.h"
#include "ss2d_launch.h"
#include "ss2d_norm_launch.h"

namespace {

constexpr int kNormMaxD = 8192;
// the backward in one cluster: its CTAs, rows to a team, and columns whose sums fit beside the teams' in 48 KB
constexpr int kClusterCtas = 8, kClusterRows = 2, kClusterD = 1536;

struct NormCall {
    ss2d::NormParams p;
    int dtype, r_dtype;
};

int norm_validate(const NormCall &c)
{
    const ss2d::NormParams &p = c.p;
    if (p.rows < 0 || p.D < 0 || p.D > kNormMaxD || p.group < 1 || p.rows > (1LL << 40))
        return SS2D_ERR_SHAPE;
    if (c.dtype != SS2D_F32 && c.dtype != SS2D_BF16 && c.dtype != SS2D_F16)
        return SS2D_ERR_DTYPE;
    if (c.r_dtype != SS2D_F32 && c.r_dtype != c.dtype)
        return SS2D_ERR_DTYPE;
    if (p.post < 0 || p.post > 2 || p.pre < 0 || p.pre > 2 || !(p.eps >= 0.f))
        return SS2D_ERR_NORM;
    const long long row = (long long)p.group * p.D;
    if (p.xs < row || (p.z && p.zs < row))
        return SS2D_ERR_STRIDE;
    return SS2D_OK;
}

bool on_device(const void *q, int dev)
{
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, q) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return (a.type == cudaMemoryTypeDevice && a.device == dev) || a.type == cudaMemoryTypeManaged;
}

int check(const void *const *need, int nneed, const void *const *opt, int nopt, const NormCall &c)
{
    for (int i = 0; i < nneed; ++i)
        if (!need[i])
            return SS2D_ERR_NULL;
    for (int i = 0; i < nneed + nopt; ++i) {
        const void *q = i < nneed ? need[i] : opt[i - nneed];
        if (q && ((uintptr_t)q & 15u) != 0)
            return SS2D_ERR_ALIGN;
    }
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        ss2d::record_error("cudaGetDevice", e);
        return SS2D_ERR_CUDA;
    }
    for (int i = 0; i < nneed + nopt; ++i) {
        const void *q = i < nneed ? need[i] : opt[i - nneed];
        if (q && !on_device(q, dev))
            return SS2D_ERR_PTR;
    }
    return SS2D_OK;
}

// Vectors where every row of every tensor starts on a 16-byte boundary, single
// values otherwise; E values a thread, in teams of the smallest power of two that
// holds a row.  Rows that fill their teams, of 8 * 2^k values or 12 * 2^k (a width of 192
// in teams of 16, not of 32 with a quarter idle), have kernels for five combinations of
// parts: a norm with or without its gate, a residual, alone or scaled and with
// biases, with the next norm, everything without biases.  The others look up what they
// have (a layer norm of 25088 rows of 192 with its bias 14.3 us against 10.2 without, backward
// 41 against 27; every part of 12544 rows of 1024 55 against 45, backward 125 against 80).
ss2d::NormPlan norm_plan(NormCall &c, bool bwd)
{
    using namespace ss2d;
    NormParams &p = c.p;
    const int esz = c.dtype == SS2D_F32 ? 4 : 2;
    const bool vec = p.D % 8 == 0 && p.xs * esz % 16 == 0 && (!p.z || p.zs * esz % 16 == 0);
    NormPlan pl{vec ? 8 : 1, p.D <= 4096 ? 8 : 16, kNormAny};
    auto team = [&](int E) {
        int t = 1;
        while (t * E < p.D)
            t <<= 1;
        return t;
    };
    if (vec && p.D <= 4096) {
        // in the backward pass r is r', which the second norm reads; the residual itself costs nothing
        const bool res = bwd ? p.pre != kNormNone : p.r != nullptr;
        const bool bias = (p.post && p.b_post) || (p.pre && p.b_pre) || p.cols >> 3;
        const int has = (p.post ? kHasPost : 0) | (p.z ? kHasGate : 0) | (res ? kHasRes : 0) |
                        (p.pre ? kHasPre : 0) | (p.s ? kHasScale : 0) | (bias ? kHasBias : 0);
        const bool known = has == kHasPost || has == (kHasPost | kHasGate) || has == (kHasRes | kHasPre) ||
                           has == (kHasRes | kHasPre | kHasScale | kHasBias) ||
                           has == (kHasPost | kHasGate | kHasRes | kHasPre | kHasScale);
        if (known && team(8) * 8 == p.D && team(8) <= 256) {
            pl.M = has;
        } else if (known && team(12) * 12 == p.D && team(12) <= 256) {
            pl = NormPlan{4, 12, has};
        }
    }
    p.tpr = team(pl.E);
    return pl;
}

cudaError_t launch_norm(const NormCall &c, const ss2d::NormPlan &pl, bool bwd, int grid, int threads, cudaStream_t st)
{
    const bool rf = c.r_dtype == SS2D_F32;
    switch (c.dtype) {
    case SS2D_F32:
        return ss2d::launch_norm_f32(c.p, pl, bwd, grid, threads, st);
    case SS2D_BF16:
        return ss2d::launch_norm_bf16(c.p, pl, bwd, rf, grid, threads, st);
    default:
        return ss2d::launch_norm_f16(c.p, pl, bwd, rf, grid, threads, st);
    }
}

}  // namespace

extern "C" {

int block_norm_fwd(const void *x, const void *z, const void *r, const float *s, const float *w_post,
                   const float *b_post, const float *w_pre, const float *b_pre, void *r_out, void *y,
                   long long rows, int D, int group, long long x_stride, long long z_stride, int post, int pre,
                   float eps, int dtype, int r_dtype, void *stream)
{
    NormCall c{};
    c.dtype = dtype;
    c.r_dtype = r_dtype;
    ss2d::NormParams &p = c.p;
    p.x = x;
    p.z = z;
    p.r = r;
    p.s = s;
    p.w_post = w_post;
    p.b_post = b_post;
    p.w_pre = w_pre;
    p.b_pre = b_pre;
    p.r_out = r_out;
    p.y = y;
    p.rows = rows;
    p.D = D;
    p.group = group;
    p.xs = x_stride;
    p.zs = z_stride;
    p.post = post;
    p.pre = pre;
    p.eps = eps;
    int rc = norm_validate(c);
    if (rc != SS2D_OK || rows == 0 || D == 0)
        return rc;
    const void *need[] = {x, r_out, pre ? y : x};
    const void *opt[] = {z, r, s, w_post, b_post, w_pre, b_pre};
    rc = check(need, 3, opt, 7, c);
    if (rc != SS2D_OK)
        return rc;
    const ss2d::NormPlan pl = norm_plan(c, false);
    const int threads = p.tpr > 256 ? p.tpr : 256;
    const long long teams = threads / p.tpr, ctas = (rows + teams - 1) / teams;
    // four CTAs of 256 threads to an SM, as many as forms of up to 64 registers run at once (302592 rows of 64 with a
    // gate: 22 us for 18.1 us of bytes).  The others, up to 128 registers with every part, run two or three and the rest
    // as a second wave (25088 rows of 192, residual and next norm, 96 registers: 13.2 us for 9.0 us of bytes)
    const int grid = ctas > 148 * 4 ? 148 * 4 : (int)ctas;
    const cudaError_t e = launch_norm(c, pl, false, grid, threads, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        ss2d::record_error("kernel launch", e);
        return SS2D_ERR_CUDA;
    }
    return SS2D_OK;
}

int block_norm_bwd(const void *x, const void *z, const void *r_out, const float *s, const float *w_post,
                   const float *b_post, const float *w_pre, const void *dr_out, const void *dy, void *dx, void *dz,
                   void *dr, float *ds, float *dw_post, float *db_post, float *dw_pre, float *db_pre,
                   long long rows, int D, int group, long long x_stride, long long z_stride, int post, int pre,
                   float eps, int dtype, int r_dtype, void *stream)
{
    NormCall c{};
    c.dtype = dtype;
    c.r_dtype = r_dtype;
    ss2d::NormParams &p = c.p;
    p.x = x;
    p.z = z;
    p.r = r_out;
    p.s = s;
    p.w_post = w_post;
    p.b_post = b_post;
    p.w_pre = w_pre;
    p.dr_out = dr_out;
    p.dy = dy;
    p.dx = dx;
    p.dz = dz;
    p.dr = dr;
    p.rows = rows;
    p.D = D;
    p.group = group;
    p.xs = x_stride;
    p.zs = z_stride;
    p.post = post;
    p.pre = pre;
    p.eps = eps;
    int rc = norm_validate(c);
    if (rc != SS2D_OK || D == 0)
        return rc;
    // column sums of a part that the call does not have are not written
    const ss2d::NormSums out{{s ? ds : nullptr, post ? dw_post : nullptr, pre ? dw_pre : nullptr,
                              post ? db_post : nullptr, pre ? db_pre : nullptr}};
    for (int i = 0; i < ss2d::kNormCols; ++i)
        p.cols |= (out.out[i] ? 1 : 0) << i;
    const void *sums[] = {out.out[0], out.out[1], out.out[2], out.out[3], out.out[4]};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (rows == 0) {
        rc = check(nullptr, 0, sums, 5, c);
        for (int i = 0; i < ss2d::kNormCols && rc == SS2D_OK && e == cudaSuccess; ++i)
            if (out.out[i])
                e = cudaMemsetAsync(out.out[i], 0, sizeof(float) * D, st);
        if (rc == SS2D_OK && e != cudaSuccess) {
            ss2d::record_error("cudaMemsetAsync", e);
            return SS2D_ERR_CUDA;
        }
        return rc;
    }
    const void *need[] = {x, dx, pre ? r_out : x, pre ? dy : x, pre ? x : dr_out, z ? dz : x};
    const void *opt[] = {z, s, w_post, b_post, w_pre, dr_out, dr, ds, dw_post, db_post, dw_pre, db_pre};
    rc = check(need, 6, opt, 12, c);
    if (rc != SS2D_OK)
        return rc;
    if (!z)
        p.dz = nullptr;
    const ss2d::NormPlan pl = norm_plan(c, true);
    int threads = p.tpr > 256 ? p.tpr : 256;
    auto count = [&](int n) { return (rows + n / p.tpr - 1) / (n / p.tpr); };   // CTAs of n threads, a row to a team
    // CTAs that the kernel's registers let onto an SM; more of them only add partials
    const int fill = 148 * (pl.M == ss2d::kNormAny ? 2 : ss2d::norm_bwd_ctas(pl.E));
    int grid = (int)(count(threads) < fill ? count(threads) : fill);
    // Few rows: one cluster of up to eight CTAs, which adds up its CTAs' sums in their shared memory; no scratch and
    // no second launch.  With a row to a team (16 of 191 float32 values: 10.2 -> 9.0 us) the device gains too; up to
    // two rows, in CTAs of 512 threads where the kernel has them, only the host does (197 rows: 9.9 -> 13.2 us in a
    // graph, but a call from Python 25.6 -> 20.3); with four rows the device took 18.7 us.
    if (p.cols && p.D <= kClusterD && grid > kClusterCtas && pl.M == ss2d::kNormAny)
        threads = 512;
    const bool cluster = p.cols && p.D <= kClusterD && count(threads) <= kClusterCtas * kClusterRows;
    if (cluster)
        grid = (int)(count(threads) < kClusterCtas ? count(threads) : kClusterCtas);
    else if (p.tpr <= 256)
        threads = 256;
    for (int i = 0; i < ss2d::kNormCols; ++i)
        p.sums[i] = out.out[i];
    void *part = nullptr;
    if (p.cols && !cluster) {
        rc = ss2d::scratch_alloc(&part, sizeof(float) * ss2d::kNormCols * grid * (size_t)D, st);
        if (rc != SS2D_OK)
            return rc;
    }
    p.part = static_cast<float *>(part);
    e = launch_norm(c, pl, true, grid, threads, st);
    if (e == cudaSuccess && part) {
        e = ss2d::launch_norm_colsum(p.part, out, grid, D, st);
    }
    cudaError_t ef = cudaSuccess;
    if (part)
        ef = cudaFreeAsync(part, st);
    if (e != cudaSuccess || ef != cudaSuccess) {
        ss2d::record_error(e != cudaSuccess ? "kernel launch" : "cudaFreeAsync", e != cudaSuccess ? e : ef);
        return SS2D_ERR_CUDA;
    }
    return SS2D_OK;
}

}  // extern "C"
