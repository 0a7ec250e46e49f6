// ss2d_delta.cu -- the C ABI of the gated delta rule (include/ss2d.h):
// argument checks, scratch and the choice between the token-by-token kernel
// and the chunked ones.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "ss2d.h"
#include "ss2d_delta_launch.h"
#include "ss2d_launch.h"

namespace {

using ss2d::DeltaParams;
using ss2d::DeltaPlan;
using ss2d::kDeltaC;

// Calls whose sequences are known to be this short go token by token.
constexpr int kRecurLen = 4;

// Segments of a long chain: CTAs that they should make, and chunks that each has at least
constexpr int kSegmentCtas = 148;
constexpr int kSegmentMin = 8;

struct Call {
    DeltaParams p;
    int dtype;
    cudaStream_t st;
};

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

int validate(const Call &c)
{
    const DeltaParams &p = c.p;
    if (p.nseq < 0 || p.L < 0 || p.L > INT_MAX - kDeltaC || p.HK < 0 || p.H < 0 || p.H > 65535)
        return SS2D_ERR_SHAPE;
    if (c.dtype != SS2D_F32 && c.dtype != SS2D_BF16 && c.dtype != SS2D_F16)
        return SS2D_ERR_DTYPE;
    if ((p.HK == 0 ? p.H != 0 : p.H % p.HK != 0) || p.DK < 16 || p.DK > ss2d::kDeltaMaxDK || p.DK % 16 != 0 ||
        p.DV < 16 || p.DV > ss2d::kDeltaMaxDV || p.DV % 16 != 0)
        return SS2D_ERR_HEADS;
    if (p.qs < (long long)p.HK * p.DK || p.ks < (long long)p.HK * p.DK || p.vs < (long long)p.H * p.DV)
        return SS2D_ERR_STRIDE;
    return SS2D_OK;
}

// Every pointer of `need` is given; those and `opt` are aligned device memory; token strides keep rows aligned.
// Bit i of `words`: pointer i, of need and then opt, is read or written value by value and may start at any of them
// (g of one token out of a sequence's)
int check(const Call &c, const void *const *need, int nneed, const void *const *opt, int nopt, unsigned words)
{
    const int esz = c.dtype == SS2D_F32 ? 4 : 2;
    for (int i = 0; i < nneed; ++i)
        if (!need[i])
            return SS2D_ERR_NULL;
    for (int i = 0; i < nneed + nopt; ++i)
        if (((uintptr_t)(i < nneed ? need[i] : opt[i - nneed]) & (words >> i & 1 ? 3u : 15u)) != 0)
            return SS2D_ERR_ALIGN;
    if (c.p.qs * esz % 16 != 0 || c.p.ks * esz % 16 != 0 || c.p.vs * esz % 16 != 0)
        return SS2D_ERR_ALIGN;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        ss2d::record_error("cudaGetDevice", e);
        return SS2D_ERR_CUDA;
    }
    for (int i = 0; i < nneed + nopt; ++i) {
        const void *q = i < nneed ? need[i] : opt[i - nneed];
        if (!q)
            continue;
        cudaPointerAttributes a;
        e = cudaPointerGetAttributes(&a, q);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return SS2D_ERR_PTR;
        }
        if (!(a.type == cudaMemoryTypeDevice && a.device == dev) && a.type != cudaMemoryTypeManaged)
            return SS2D_ERR_PTR;
    }
    return SS2D_OK;
}

int run(Call &c, const DeltaPlan &pl, int what)
{
    cudaError_t e;
    switch (c.dtype) {
    case SS2D_BF16:
        e = what == ss2d::kDeltaBwd ? ss2d::launch_delta_bwd_bf16(c.p, pl, c.st)
                                    : ss2d::launch_delta_bf16(c.p, pl, what, c.st);
        break;
    case SS2D_F16:
        e = what == ss2d::kDeltaBwd ? ss2d::launch_delta_bwd_f16(c.p, pl, c.st)
                                    : ss2d::launch_delta_f16(c.p, pl, what, c.st);
        break;
    default:
        e = what == ss2d::kDeltaBwd ? ss2d::launch_delta_bwd_f32(c.p, pl, c.st)
                                    : ss2d::launch_delta_f32(c.p, pl, what, c.st);
        break;
    }
    if (e != cudaSuccess) {
        ss2d::record_error("kernel launch", e);
        return SS2D_ERR_CUDA;
    }
    return SS2D_OK;
}

// the chunked passes, with their scratch
int run_chunked(Call &c, bool bwd)
{
    DeltaParams &p = c.p;
    DeltaPlan pl;
    pl.dkp = p.DK <= 64 ? 64 : 128;
    pl.npi = c.dtype == SS2D_F32 ? 3 : c.dtype == SS2D_F16 ? 2 : 1;
    pl.np = bwd || p.h_last || c.dtype == SS2D_F32 ? 3 : 2;
    pl.npp = bwd || c.dtype == SS2D_F32 ? 3 : 2;
    p.NC = (p.L + kDeltaC - 1) / kDeltaC;
    p.nslots = p.cu ? p.T / kDeltaC + p.nseq : (long long)p.nseq * p.NC;
    if (p.nslots > INT_MAX || p.HK > 65535)
        return SS2D_ERR_SHAPE;
    // Few long chains are cut into segments of SC chunks, about one for each SM that
    // a CTA of 64 DV columns can have, when at least four to a chain come of it: the
    // segments run twice and their states are followed one by one.
    const long long ctas = (long long)((p.DV + 63) / 64) * p.H;
    const long long sc = (p.nslots * ctas + kSegmentCtas - 1) / kSegmentCtas;
    if (ctas * p.nseq * 4 <= kSegmentCtas && p.nslots >= 4LL * kSegmentMin * p.nseq)
        p.SC = (int)(sc < kSegmentMin ? kSegmentMin : sc);
    const size_t segs = !p.SC ? 0 : p.cu ? p.nslots / p.SC + p.nseq
                                         : (size_t)p.nseq * ((p.NC + p.SC - 1) / p.SC);
    const size_t n = (size_t)p.nslots, nh = n * p.H, part = ss2d::kTriBytes;
    // float16 chains read k and q as they are, but for the outputs of few wide heads
    const bool parts = c.dtype == SS2D_F32 ||
                       (c.dtype == SS2D_F16 && !bwd && pl.dkp == 128 && ss2d::delta_split_f16(p));
    const size_t kp = parts ? n * p.HK * pl.npi * kDeltaC * pl.dkp * 2 : 0;
    const size_t sx = bwd ? nh * p.DV * pl.dkp * 4 : 0, vx = bwd ? nh * p.DV * kDeltaC * 4 : 0;
    const size_t ns = segs * p.H * p.DV * pl.dkp * 4;
    const size_t size[] = {kp, kp, nh * pl.np * part, nh * pl.npp * part, nh * ss2d::kDeltaVec * 4, sx, sx, vx, vx, ns, ns, bwd ? ns : 0, bwd ? ns : 0,
                           segs * p.H * 3 * pl.dkp * pl.dkp * 2};
    size_t off[14], total = 0;
    for (int i = 0; i < 14; ++i) {
        off[i] = total;
        total += up256(size[i]);
    }
    void *scratch = nullptr;
    int rc = ss2d::scratch_alloc(&scratch, total, c.st);
    if (rc != SS2D_OK)
        return rc;
    char *b = static_cast<char *>(scratch);
    auto f = [&](int i) { return reinterpret_cast<float *>(b + off[i]); };
    p.kp = parts ? b + off[0] : nullptr;
    p.qp = parts ? b + off[1] : nullptr;
    p.Tp = b + off[2];
    p.Pp = b + off[3];
    p.vec = f(4);
    p.Sx = f(5);
    p.dSx = f(6);
    p.Vx = f(7);
    p.dXx = f(8);
    p.Ns = f(9);
    p.Sin = f(10);
    p.dNs = f(11);
    p.dSin = f(12);
    p.Ms = b + off[13];
    rc = run(c, pl, bwd ? ss2d::kDeltaBwd : ss2d::kDeltaFwd);
    const cudaError_t e = cudaFreeAsync(scratch, c.st);
    if (rc == SS2D_OK && e != cudaSuccess) {
        ss2d::record_error("cudaFreeAsync", e);
        return SS2D_ERR_CUDA;
    }
    return rc;
}

}  // namespace

extern "C" {

int gated_delta_rule_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *h0, void *o, float *h_last, const int *cu_seqlens, int nseq, int L, int HK,
                         int H, int DK, int DV, long long q_stride, long long k_stride, long long v_stride,
                         float scale, int reverse, int dtype, void *stream)
{
    Call c{};
    DeltaParams &p = c.p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.h0 = h0;
    p.o = o;
    p.h_last = h_last;
    p.cu = cu_seqlens;
    p.nseq = nseq;
    p.L = L;
    p.HK = HK;
    p.H = H;
    p.DK = DK;
    p.DV = DV;
    p.qs = q_stride;
    p.ks = k_stride;
    p.vs = v_stride;
    p.scale = scale;
    p.reverse = reverse ? 1 : 0;
    p.T = cu_seqlens ? L : (long long)nseq * L;
    c.dtype = dtype;
    c.st = static_cast<cudaStream_t>(stream);
    int rc = validate(c);
    if (rc != SS2D_OK || nseq == 0 || H == 0 || (p.T == 0 && !h_last))
        return rc;
    const void *opt[] = {h0, h_last, cu_seqlens};
    const void *need[] = {q, k, v, g, beta, o};
    const unsigned words = 1 << 3 | 1 << 4 | 1 << 8;   // g, beta, cu_seqlens
    rc = p.T ? check(c, need, 6, opt, 3, words) : check(c, nullptr, 0, opt, 3, words >> 6);
    if (rc != SS2D_OK)
        return rc;
    if (L <= kRecurLen)
        return run(c, DeltaPlan{}, ss2d::kDeltaRecur);
    return run_chunked(c, false);
}

int gated_delta_rule_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                         const float *h0, const void *dout, const float *dh_last, void *dq, void *dk, void *dv,
                         float *dg, float *dbeta, float *dh0, const int *cu_seqlens, int nseq, int L, int HK, int H,
                         int DK, int DV, long long q_stride, long long k_stride, long long v_stride, float scale,
                         int reverse, int dtype, void *stream)
{
    Call c{};
    DeltaParams &p = c.p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.h0 = h0;
    p.dout = dout;
    p.dh_last = dh_last;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dg = dg;
    p.dbeta = dbeta;
    p.dh0 = dh0;
    p.cu = cu_seqlens;
    p.nseq = nseq;
    p.L = L;
    p.HK = HK;
    p.H = H;
    p.DK = DK;
    p.DV = DV;
    p.qs = q_stride;
    p.ks = k_stride;
    p.vs = v_stride;
    p.scale = scale;
    p.reverse = reverse ? 1 : 0;
    p.T = cu_seqlens ? L : (long long)nseq * L;
    c.dtype = dtype;
    c.st = static_cast<cudaStream_t>(stream);
    int rc = validate(c);
    if (rc == SS2D_OK && H == 0 && HK > 0)   // no kernel runs that could write dq and dk
        rc = SS2D_ERR_HEADS;
    if (rc != SS2D_OK || nseq == 0 || H == 0 || (p.T == 0 && !dh0))
        return rc;
    const void *opt[] = {h0, dh_last, dh0, cu_seqlens};
    const void *need[] = {q, k, v, g, beta, dout, dq, dk, dv, dg, dbeta};
    const unsigned words = 1 << 3 | 1 << 4 | 1 << 9 | 1 << 10 | 1 << 14;   // g, beta, dg, dbeta, cu_seqlens
    rc = p.T ? check(c, need, 11, opt, 4, words) : check(c, nullptr, 0, opt, 4, words >> 11);
    if (rc != SS2D_OK)
        return rc;
    if (p.T == 0) {   // no token anywhere: the state passes through
        const size_t bytes = (size_t)nseq * H * DK * DV * 4;
        cudaError_t e = cudaSuccess;
        if (!dh_last)
            e = cudaMemsetAsync(dh0, 0, bytes, c.st);
        else if (dh0 != dh_last)
            e = cudaMemcpyAsync(dh0, dh_last, bytes, cudaMemcpyDeviceToDevice, c.st);
        if (e != cudaSuccess) {
            ss2d::record_error("cudaMemcpyAsync", e);
            return SS2D_ERR_CUDA;
        }
        return SS2D_OK;
    }
    return run_chunked(c, true);
}

int gated_delta_rule_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                          float *state, const int *slots, void *o, int B, long long nstates, int HK, int H, int DK,
                          int DV, long long q_stride, long long k_stride, long long v_stride, float scale, int dtype,
                          void *stream)
{
    Call c{};
    DeltaParams &p = c.p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.o = o;
    p.pool = state;
    p.slots = slots;
    p.npool = nstates;
    p.nseq = B;
    p.L = 1;
    p.HK = HK;
    p.H = H;
    p.DK = DK;
    p.DV = DV;
    p.qs = q_stride;
    p.ks = k_stride;
    p.vs = v_stride;
    p.scale = scale;
    p.T = B;
    c.dtype = dtype;
    c.st = static_cast<cudaStream_t>(stream);
    int rc = validate(c);
    if (rc != SS2D_OK)
        return rc;
    if (nstates < 0 || (!slots && nstates < B))
        return SS2D_ERR_SHAPE;
    if (B == 0 || H == 0)
        return SS2D_OK;
    // a pool of no states: every slot is skipped, the pointer is not read
    const void *need[] = {q, k, v, g, beta, o, nstates ? state : o};
    rc = check(c, need, 7, reinterpret_cast<const void *const *>(&slots), 1, 1 << 3 | 1 << 4 | 1 << 7);   // g, beta, slots
    if (rc != SS2D_OK)
        return rc;
    if (!p.pool)
        p.pool = static_cast<float *>(o);
    return run(c, DeltaPlan{}, ss2d::kDeltaRecur);
}

}  // extern "C"
