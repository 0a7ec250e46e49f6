"""The block norms (block_norm_fwd, block_norm_bwd): the float64 oracle against
central differences, the refusals, and the CUDA kernels against the oracle.

Tolerances of the GPU tests, per element.  The kernels compute in float32 and
round once on store: half a step of the stored type, eps(t) / 2 * |ref|, plus
the float32 arithmetic.  That is a sum over a row by a tree whose longest
path is E + log2(TPR) + TPR / 32 <= 16 + 9 + 16 additions and at most 20
operations on each value, each off by 2^-24 of a quantity no larger than the
row's largest (M, below): F32 = 64 * 2^-24 * M.  Column sums over rows add
one value per visited row, then teams (<= 64), partials (<= 444 / 32) and 32
runs by a tree: at most (rows + 128) additions, and 32 operations on each term:
(rows + 160) * 2^-24 * sum |term|."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import block_norm_np as onp
from selective_scan_ss2d_b200 import binding, build

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def make(rows, D, post="rms", pre="rms", gate=True, res=True, scale=True, bias=True, seed=0):
    rng = np.random.default_rng([seed, rows, D])
    a = dict(x=1.5 * rng.standard_normal((rows, D)) + 0.3, post=post, pre=pre)
    a["z"] = rng.standard_normal((rows, D)) if gate else None
    a["r"] = 2.0 * rng.standard_normal((rows, D)) if res else None
    a["s"] = 0.1 + 0.3 * rng.standard_normal(D) if scale else None
    for n, on in (("post", post != "none"), ("pre", pre != "none")):
        a["w_" + n] = 1.0 + 0.2 * rng.standard_normal(D) if on else None
        a["b_" + n] = 0.2 * rng.standard_normal(D) if on and bias else None
    return a


COMBOS = [("rms", "rms"), ("layer", "layer"), ("none", "layer"), ("rms", "none"), ("none", "none"), ("layer", "rms")]


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("post,pre", COMBOS)
@pytest.mark.parametrize("gate,scale", [(True, True), (False, False)])
def test_oracle_gradients_against_differences(post, pre, gate, scale):
    a = make(3, 7, post, pre, gate, True, scale, True)
    rng = np.random.default_rng(5)
    dr_out, dy = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))

    def loss(**k):
        r_out, y = onp.block_norm_fwd(**{**a, **k})
        return (dr_out * r_out).sum() + (0.0 if y is None else (dy * y).sum())

    r_out, _ = onp.block_norm_fwd(**a)
    g = onp.block_norm_bwd(a["x"], dr_out, dy if pre != "none" else None, r_out=r_out, z=a["z"], s=a["s"], post=post,
                           w_post=a["w_post"], b_post=a["b_post"], pre=pre, w_pre=a["w_pre"])
    for name in ("x", "z", "r", "s", "w_post", "b_post", "w_pre", "b_pre"):
        if a[name] is None:
            continue
        num, h = np.zeros_like(a[name]), 1e-5
        for i in np.ndindex(a[name].shape):
            hi, lo = a[name].copy(), a[name].copy()
            hi[i] += h
            lo[i] -= h
            num[i] = (loss(**{name: hi}) - loss(**{name: lo})) / (2 * h)
        # truncation h^2 |f'''| / 6 and rounding 2^-53 |f| / h, both below 1e-8 at these sizes
        np.testing.assert_allclose(g["d" + name], num, rtol=1e-6, atol=1e-7, err_msg=name)


def test_oracle_norms_by_hand():
    x = np.array([[3.0, -3.0, 3.0, -3.0]])
    assert np.allclose(onp.norm(x, "rms", 0.0)[0], [[1, -1, 1, -1]])
    assert np.allclose(onp.norm(x + 5, "layer", 0.0)[0], [[1, -1, 1, -1]])
    assert np.allclose(onp.norm(x, "rms", 7.0)[0], x / 4.0)


# ---------------------------------------------------------------- refusals
def _fwd(lib, p, rows=2, D=8, group=1, xs=8, zs=8, post=1, pre=1, eps=1e-5, dtype=1, rdt=0, nulls=()):
    a = [p] * 10
    for i in nulls:
        a[i] = None
    return lib.block_norm_fwd(*a, rows, D, group, xs, zs, post, pre, eps, dtype, rdt, None)


def _bwd(lib, p, rows=2, D=8, group=1, xs=8, zs=8, post=1, pre=1, eps=1e-5, dtype=1, rdt=0, nulls=()):
    a = [p] * 17
    for i in nulls:
        a[i] = None
    return lib.block_norm_bwd(*a, rows, D, group, xs, zs, post, pre, eps, dtype, rdt, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_argument_errors_are_reported_without_cuda(lib, call):
    buf = (ctypes.c_float * 64)()
    addr = ctypes.addressof(buf)
    p = ctypes.c_void_p(addr + (-addr) % 16)
    assert call(lib, p, rows=-1) == -2
    assert call(lib, p, D=8200, xs=8200, zs=8200) == -2
    assert call(lib, p, D=-8) == -2
    assert call(lib, p, group=0) == -2
    assert call(lib, p, dtype=3) == -3
    assert call(lib, p, dtype=1, rdt=2) == -3
    assert call(lib, p, post=3) == -12
    assert call(lib, p, pre=-1) == -12
    assert call(lib, p, eps=-1.0) == -12
    assert call(lib, p, eps=float("nan")) == -12
    assert call(lib, p, xs=7) == -13
    assert call(lib, p, group=2, xs=15, zs=16) == -13
    assert call(lib, p, group=2, xs=16, zs=8) == -13
    assert call(lib, p, nulls=(0,)) == -1
    assert call(lib, p, D=0, xs=0, zs=0, nulls=range(10)) == 0
    assert call(lib, ctypes.c_void_p(p.value + 4)) == -6
    for st in (-12, -13):
        assert binding.ss2d_status_string(st) != "unknown status"


def test_missing_parts_are_reported(lib):
    buf = (ctypes.c_float * 64)()
    addr = ctypes.addressof(buf)
    p = ctypes.c_void_p(addr + (-addr) % 16)
    assert _fwd(lib, p, nulls=(8,)) == -1          # r_out
    assert _fwd(lib, p, nulls=(9,)) == -1          # y with a pre norm
    assert _fwd(lib, p, rows=0, nulls=range(10)) == 0
    assert _bwd(lib, p, nulls=(2,)) == -1          # r' with a pre norm
    assert _bwd(lib, p, nulls=(8,)) == -1          # dy with a pre norm
    assert _bwd(lib, p, pre=0, nulls=(7,)) == -1   # dr_out without one
    assert _bwd(lib, p, nulls=(9,)) == -1          # dx
    assert _bwd(lib, p, nulls=(10,)) == -1         # dz with a gate


def test_binding_validates_tensors(lib):
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensors only"):
        binding.block_norm_fwd(x)
    with pytest.raises(ValueError, match="post and pre"):
        binding.block_norm_fwd(x, post="group")
    with pytest.raises(TypeError):
        binding.block_norm_fwd(x.double())
    with pytest.raises(ValueError, match="device tensors only"):
        binding.block_norm_bwd(x, x)


# --------------------------------------------------------------------- GPU
def dev(a, dtype, rdt):
    """the case's arrays on the device, and the float64 values that they hold"""
    t, f = {}, {}
    for n, v in a.items():
        if v is None or isinstance(v, str):
            t[n] = f[n] = v
            continue
        dt = DT[dtype] if n in ("x", "z") else DT[rdt] if n == "r" else torch.float32
        t[n] = torch.from_numpy(np.ascontiguousarray(v)).to(dt).cuda()
        f[n] = t[n].double().cpu().numpy()
    return t, f


def near(got, ref, dt, M, what):
    got = got.double().cpu().numpy()
    half = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    tiny = torch.finfo(dt).tiny   # below it, steps are absolute
    bound = half * np.maximum(np.abs(ref), tiny) + 64 * U * M
    err = np.abs(got - ref)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.2f} of the bound"


def rowmax(*arrays):
    return sum(np.abs(v).max(-1, keepdims=True) for v in arrays if v is not None)


SHAPES = [(1, 1), (70, 96), (41, 768), (3, 5), (7, 8), (9, 64), (33, 96), (65, 191), (130, 192), (17, 384), (5, 1000), (12, 1024),
          (6, 4096), (3, 4100), (2, 8192)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dtype,rdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
def test_forward_and_backward_match_oracle(rows, D, dtype, rdt):
    post, pre = COMBOS[(rows + D) % len(COMBOS)]
    check(make(rows, D, post, pre), dtype, rdt)


@pytest.mark.gpu
@pytest.mark.parametrize("post,pre", COMBOS)
@pytest.mark.parametrize("gate,res,scale,bias", [(True, True, True, True), (False, False, False, False),
                                                 (True, False, False, True), (False, True, True, False)])
def test_every_combination_of_parts(post, pre, gate, res, scale, bias):
    check(make(37, 72, post, pre, gate, res, scale, bias), "bf16", "f32" if res else "bf16")
    check(make(29, 64, post, pre, gate, res, scale, bias), "f16", "f16")    # rows that fill their teams
    check(make(21, 192, post, pre, gate, res, scale, bias), "bf16", "bf16")
    check(make(11, 45, post, pre, gate, res, scale, bias), "f32", "f32")


def check(a, dtype, rdt, seed=1):
    t, f = dev(a, dtype, rdt)
    rt = DT[rdt] if a["r"] is not None else DT[dtype]
    r_out, y = binding.block_norm_fwd(**t)
    torch.cuda.synchronize()
    ref_r, ref_y = onp.block_norm_fwd(**f)
    tn = onp.branch(f["x"], f["z"], f["s"], f["post"], f["w_post"], f["b_post"], 1e-5)
    # quantities of a row: the normalised branch, the residual, and what the norm makes of their errors
    M = rowmax(tn[0], tn[2], tn[3], ref_r, f["r"])
    near(r_out, ref_r, rt, M, "r_out")
    assert r_out.dtype == rt
    if y is not None:
        n2, rs2 = onp.norm(ref_r, f["pre"], 1e-5)
        wmax = 1.0 if f["w_pre"] is None else np.abs(f["w_pre"]).max()
        near(y, ref_y, DT[dtype], (M * rs2 * (1 + np.abs(n2).max(-1, keepdims=True)) + rowmax(n2)) * wmax
             + rowmax(ref_y, f["b_pre"][None] if f["b_pre"] is not None else None), "y")
    rng = np.random.default_rng(seed)
    dr = torch.from_numpy(rng.standard_normal(a["x"].shape)).to(rt).cuda()
    dy = torch.from_numpy(rng.standard_normal(a["x"].shape)).to(DT[dtype]).cuda() if y is not None else None
    kw = {n: t[n] for n in ("z", "s", "post", "w_post", "b_post", "pre", "w_pre", "b_pre")}
    g = binding.block_norm_bwd(t["x"], dr, dy, r_out=r_out, residual=a["r"] is not None, **kw)
    torch.cuda.synchronize()
    fr, fdy = r_out.double().cpu().numpy(), dy.double().cpu().numpy() if dy is not None else None
    fdr = dr.double().cpu().numpy()
    ref = onp.block_norm_bwd(f["x"], fdr, fdy, r_out=fr, z=f["z"], s=f["s"], post=f["post"], w_post=f["w_post"],
                             b_post=f["b_post"], pre=f["pre"], w_pre=f["w_pre"])
    MG = rowmax(fdr)
    if fdy is not None:
        n2, rs2 = onp.norm(fr, f["pre"], 1e-5)
        wd = fdy * (1.0 if f["w_pre"] is None else f["w_pre"])
        # |d|, |n| mean|d n| and the centred value's own error (|r'| rs against n)
        big = np.abs(n2).max(-1, keepdims=True)
        MG = MG + rs2 * rowmax(wd) * (1 + big + big * big) * (1 + rowmax(fr) * rs2)
    if a["r"] is not None:
        near(g["dr"], ref["dr"], rt, MG, "dr")
    else:
        assert g["dr"] is None
    sm = 1.0 if f["s"] is None else np.abs(f["s"]).max()
    zm = 1.0 + (0.0 if f["z"] is None else np.abs(f["z"]).max(-1, keepdims=True))
    n, rs, p, _ = tn
    rel = 1.0   # the normalised branch's own error, against its size
    if f["post"] != "none":
        rel = 1 + rowmax(f["x"]) * rs
    if f["z"] is not None:
        near(g["dz"], ref["dz"], DT[dtype], MG * sm * rowmax(p) * zm * rel, "dz")
    Mp = MG * sm * zm
    if f["post"] != "none":
        wp = 1.0 if f["w_post"] is None else np.abs(f["w_post"]).max()
        big = rowmax(n)
        Mp = rs * wp * Mp * (1 + big + big * big) * rel
    near(g["dx"], ref["dx"], DT[dtype], Mp, "dx")
    rows = a["x"].shape[0]
    # a term's relative error: its factors', bounded by what G, n and t were bounded by, against their sizes
    for name in ("ds", "dw_post", "db_post", "dw_pre", "db_pre"):
        want = {"ds": f["s"], "dw_post": f["w_post"], "db_post": f["b_post"], "dw_pre": f["w_pre"],
                "db_pre": f["b_pre"]}[name]
        if want is None:
            assert g[name] is None
            continue
        got = g[name].double().cpu().numpy()
        term = {"ds": MG * rowmax(tn[3]) * rel, "dw_post": MG * sm * zm * rowmax(n) * rel, "db_post": MG * sm * zm,
                "dw_pre": rowmax(fdy) * rowmax(n2) * (1 + rowmax(fr) * rs2) if fdy is not None else 0,
                "db_pre": rowmax(fdy) if fdy is not None else 0}[name]
        bound = (rows + 160) * U * ref["abs"][name] + 64 * U * np.sum(term)
        err = np.abs(got - ref[name])
        assert np.all(err <= bound), f"{name}: {np.max(err / bound):.2f} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("rows,D,post,pre", [(64, 191, "rms", "none"), (256, 191, "layer", "rms"), (257, 191, "rms", "none"),
                                             (512, 64, "rms", "none"), (513, 64, "none", "layer"), (16, 1536, "rms", "layer"),
                                             (33, 1536, "rms", "none"), (5, 1544, "layer", "layer")])
def test_column_sums_on_both_sides_of_one_cluster(rows, D, post, pre):
    for bias in (False, True):
        check(make(rows, D, post, pre, gate=True, res=pre != "none", scale=pre != "none", bias=bias), "bf16", "bf16")


@pytest.mark.gpu
def test_many_rows_and_repeatable_sums():
    a = make(5003, 200)
    check(a, "bf16", "f32")
    t, _ = dev(a, "bf16", "f32")
    r_out, _ = binding.block_norm_fwd(**t)
    kw = {n: t[n] for n in ("z", "s", "post", "w_post", "b_post", "pre", "w_pre", "b_pre")}
    one = binding.block_norm_bwd(t["x"], r_out, t["x"], r_out=r_out, **kw)
    two = binding.block_norm_bwd(t["x"], r_out, t["x"], r_out=r_out, **kw)
    for n in binding.NORM_GRAD_NAMES:
        assert torch.equal(one[n], two[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("off", [0, 8, 3])
def test_slices_of_a_projection(off):
    """x and z as (M, G, D) slices of wider rows give what their copies give."""
    M, G, D = 21, 3, 40
    gen = torch.Generator().manual_seed(off)
    wide = torch.randn(M, 2 * G * D + 16 + off, generator=gen).to(torch.bfloat16).cuda()
    x = wide[:, :G * D].unflatten(1, (G, D))
    z = wide[:, 16 + G * D:16 + 2 * G * D].unflatten(1, (G, D))
    w = torch.rand(D, generator=gen).cuda()
    one = binding.block_norm_fwd(x, z=z, post="rms", w_post=w)[0]
    two = binding.block_norm_fwd(x.contiguous(), z=z.contiguous(), post="rms", w_post=w)[0]
    three = binding.block_norm_fwd(x.contiguous(), z=z, post="rms", w_post=w)[0]
    # the vector and the single-value kernels add a row's squares in another order; both then round to bfloat16, half
    # a step (up to 2^-8 of the value) each
    far = (one.float() - two.float()).abs() - 2 ** -7 * two.float().abs() - 1e-6
    assert float(far.max()) <= 0 and torch.equal(one, three)
    g1 = binding.block_norm_bwd(x, two, z=z, post="rms", w_post=w, residual=False)
    g2 = binding.block_norm_bwd(x.contiguous(), two, z=z.contiguous(), post="rms", w_post=w, residual=False)
    for n in ("dx", "dz", "dw_post"):
        a, b = g1[n].float(), g2[n].float()
        assert float(((a - b).abs() - 2 ** -7 * b.abs() - 1e-4 * b.abs().max()).max()) <= 0, n
    with pytest.raises(ValueError, match="packed rows"):
        binding.block_norm_fwd(wide[:, ::2][:, :D])


@pytest.mark.gpu
def test_rows_past_32_bits_and_groups_of_one():
    """rows 2^24 values apart: the bits of packed ones; so are groups of one row, whatever their own stride"""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, z, d = (torch.randn(140, 64, device="cuda", generator=g).bfloat16() for _ in range(3))
    far = torch.empty(140, 1 << 24, dtype=torch.bfloat16, device="cuda")
    fx, fz = far[:, :64], far[:, 64:128]
    fx.copy_(x)
    fz.copy_(z)
    want, _ = binding.block_norm_fwd(x, z=z, post="rms")
    back = binding.block_norm_bwd(x, d, z=z, post="rms")
    for a, b, view in ((fx, fz, (140, 64)), (fx[:, None], fz[:, None], (140, 1, 64))):
        assert not a.is_contiguous()
        got, _ = binding.block_norm_fwd(a, z=b, post="rms")
        grad = binding.block_norm_bwd(a, d.view(view), z=b, post="rms")
        assert torch.equal(got.view(140, 64), want)
        assert all(torch.equal(grad[n].view(140, 64), back[n]) for n in ("dx", "dz"))


@pytest.mark.gpu
def test_in_place_residual_stream_and_capture():
    a = make(64, 192, "none", "layer")
    t, _ = dev(a, "bf16", "f32")
    ref_r, ref_y = binding.block_norm_fwd(**t)
    side = torch.cuda.Stream()
    r = t["r"].clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r1, y1 = binding.block_norm_fwd(**{**t, "r": r}, r_out=r)
    side.synchronize()
    assert torch.equal(r1, ref_r) and torch.equal(y1, ref_y) and r1.data_ptr() == r.data_ptr()
    # forward and backward captured and replayed on new inputs
    x = t["x"].clone()
    dr, dy = torch.ones_like(ref_r), torch.ones_like(ref_y)
    kw = {n: t[n] for n in ("z", "s", "post", "w_post", "b_post", "pre", "w_pre", "b_pre")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, y2 = binding.block_norm_fwd(**{**t, "x": x})
        g2 = binding.block_norm_bwd(x, dr, dy, r_out=r2, **kw)
    for f in (1.0, -0.5):
        x.copy_(t["x"] * f)
        graph.replay()
        r3, y3 = binding.block_norm_fwd(**{**t, "x": x})
        g3 = binding.block_norm_bwd(x, dr, dy, r_out=r3, **kw)
        torch.cuda.synchronize()
        assert torch.equal(r2, r3) and torch.equal(y2, y3)
        for n in binding.NORM_GRAD_NAMES:
            assert (g2[n] is None and g3[n] is None) or torch.equal(g2[n], g3[n]), n


@pytest.mark.gpu
def test_empty_and_extreme_rows():
    w = torch.ones(16, device="cuda")
    x0 = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    r0, y0 = binding.block_norm_fwd(x0, pre="rms", w_pre=w)
    assert r0.shape == y0.shape == (0, 16)
    g0 = binding.block_norm_bwd(x0, x0, x0, r_out=r0, pre="rms", w_pre=w, b_pre=w, s=w)
    assert not g0["dw_pre"].any() and not g0["db_pre"].any() and not g0["ds"].any()
    # zeros, one huge value, and a gate whose e^-z overflows: the neighbours stay as they are
    x = torch.ones(4, 16, device="cuda")
    x[0] = 0
    x[1, 3] = 1e18
    z = torch.ones(4, 16, device="cuda")
    z[2] = -200.0
    y = binding.block_norm_fwd(x, z=z, post="rms", w_post=w)[0]
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and not y[0].any() and not y[2].any()
    assert abs(float(y[1, 3]) - 4.0 / (1 + np.exp(-1.0))) < 1e-5
    x[3, 0] = float("nan")
    y = binding.block_norm_fwd(x, z=z, post="layer", w_post=w)[0]
    torch.cuda.synchronize()
    assert torch.isnan(y[3]).all() and torch.isfinite(y[:3]).all()
