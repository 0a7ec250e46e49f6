"""The block norms at the edges of what their calls allow: eps = 0 where rows
do not fill the last step's teams, and sums of parts that a call does not have."""
from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import test_block_norm as tb
from oracle import block_norm_np as onp
from selective_scan_ss2d_b200 import binding


@pytest.fixture
def no_eps(monkeypatch):
    """both sides of test_block_norm's checks with eps = 0 (their bounds' 1e-5 is a 1e-5th of the rows' variance)"""
    for mod in (binding, onp):
        for n in ("block_norm_fwd", "block_norm_bwd"):
            monkeypatch.setattr(mod, n, functools.partial(getattr(mod, n), eps=0.0))


# every kernel with a team that has no row in its last step: single values, vectors, 12 and 16 values a thread, one
# cluster and partial sums, teams of a few lanes up to several warps
EPS0 = [("bf16", 37, 40), ("f32", 37, 45), ("f16", 29, 64), ("bf16", 3001, 64), ("bf16", 21, 192), ("f32", 4003, 192),
        ("bf16", 1187, 1024), ("f32", 3, 4100), ("f16", 700, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,D", EPS0)
@pytest.mark.parametrize("post,pre,gate,scale,bias", [
    ("rms", "none", False, False, False), ("rms", "none", True, False, False), ("none", "layer", False, False, False),
    ("none", "layer", False, True, True), ("rms", "rms", True, True, False), ("layer", "layer", True, True, True)])
def test_eps_zero_with_teams_that_have_no_row(dtype, rows, D, post, pre, gate, scale, bias, no_eps):
    tb.check(tb.make(rows, D, post, pre, gate, pre != "none", scale, bias), dtype, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["rms", "layer"])
def test_gradient_of_a_length_normalisation(how):
    """q scaled to length 1 by an rms norm without eps, 360 rows of 32: the weight's gradient too"""
    rng = np.random.default_rng(11)
    x, d = (torch.from_numpy(rng.standard_normal((360, 32))).float().cuda() for _ in range(2))
    w = torch.full((32,), 32 ** -0.5, device="cuda")
    g = binding.block_norm_bwd(x, d, post=how, w_post=w, eps=0.0, residual=False)
    ref = onp.block_norm_bwd(*(t.double().cpu().numpy() for t in (x, d)), post=how, w_post=w.double().cpu().numpy(),
                             eps=0.0)
    # (360 + 160) additions and 64 operations on each term, see test_block_norm
    err = np.abs(g["dw_post"].double().cpu().numpy() - ref["dw_post"])
    assert np.all(err <= (360 + 160 + 64) * tb.U * ref["abs"]["dw_post"])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [0, 5, 5003])   # no kernel, one cluster, partial sums
@pytest.mark.parametrize("post", ["none", "rms"])
def test_sums_of_parts_that_a_call_does_not_have_are_left(rows, post):
    """the C call with every output given, and no s and no second norm: ds, dw_pre and db_pre keep what they held"""
    D, lib = 64, binding.lib()
    x, d, dx = (torch.ones(max(rows, 1), D, device="cuda") for _ in range(3))
    w = torch.ones(D, device="cuda")
    sums = {n: torch.full((D,), 7.0, device="cuda") for n in ("ds", "dw_post", "db_post", "dw_pre", "db_pre")}
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = lib.block_norm_bwd(p(x), None, None, None, p(w), None, None, p(d), None, p(dx), None, None,
                            *map(p, sums.values()), rows, D, 1, D, D, binding.NORMS[post], 0, 1e-5, 0, 0, None)
    torch.cuda.synchronize()
    assert rc == 0
    has = ("dw_post", "db_post") if post != "none" else ()
    for n, v in sums.items():
        assert bool((v != 7).all()) if n in has else bool((v == 7).all()), n


@pytest.mark.gpu
@pytest.mark.parametrize("rows,D,dtype", [(9, 64, "bf16"), (700, 191, "f32"), (5003, 192, "bf16"), (301, 4100, "f16")])
def test_gradients_in_place(rows, D, dtype):
    """dx in x's place and dr in dr_out's, as the header allows: the bits of separate ones"""
    gen = torch.Generator(device="cuda").manual_seed(D)
    dt, lib = tb.DT[dtype], binding.lib()
    x, z, r, d, dy = (torch.randn(rows, D, device="cuda", generator=gen).to(dt) for _ in range(5))
    w = torch.rand(D, device="cuda", generator=gen)
    want = binding.block_norm_bwd(x, d, dy, r_out=r, z=z, s=w, post="rms", w_post=w, pre="layer", w_pre=w, b_pre=w)
    dz, sums = torch.empty_like(z), [torch.empty_like(w) for _ in range(4)]
    p = lambda t: t.data_ptr()  # noqa: E731
    ds, dwq, dwp, dbp = sums
    rc = lib.block_norm_bwd(p(x), p(z), p(r), p(w), p(w), None, p(w), p(d), p(dy), p(x), p(dz), p(d), p(ds), p(dwq),
                            None, p(dwp), p(dbp), rows, D, 1, D, D, 1, 2, 1e-5, binding._DTYPES[dt], binding._DTYPES[dt],
                            None)
    torch.cuda.synchronize()
    assert rc == 0
    for n, v in (("dx", x), ("dr", d), ("dz", dz), ("ds", ds), ("dw_post", dwq), ("dw_pre", dwp)):
        assert torch.equal(want[n], v), n


@pytest.mark.gpu
def test_more_rows_than_32_bits_count():
    """2^31 + 8 rows of one value, in groups of two and packed: the last ones, and a column sum of all"""
    M = (1 << 30) + 4
    wide = torch.zeros(M, 4, dtype=torch.bfloat16, device="cuda")
    x = wide[:, :2].unflatten(1, (2, 1))
    x[-3:] = torch.tensor([[1.0, -2.0], [3.0, 4.0], [5.0, -6.0]], device="cuda").bfloat16()[..., None]
    s = torch.full((1,), 2.0, device="cuda")
    r, _ = binding.block_norm_fwd(x, s=s)
    assert torch.equal(r[-3:], 2 * x[-3:]) and not r[:1000].any() and not r[-1000:-3].any()
    g = binding.block_norm_bwd(x, r, s=s, residual=False)
    torch.cuda.synchronize()
    assert torch.equal(g["dx"][-3:], 2 * r[-3:]) and float(g["ds"]) == 2 * (1 + 4 + 9 + 16 + 25 + 36)
