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
