"""The gated delta rule (gated_delta_rule_fwd, _bwd, _step): the float64 oracle
against central differences and closed forms, the refusals, and the CUDA
kernels against the oracle.

Tolerances of the GPU tests, per element: half a step of the stored type on the
value, plus the arithmetic.  A chunk's results are at most six chained sums
of up to 256 products; a tensor-core sum may truncate (2^-23 of its terms),
and the errors of n terms add like sqrt(n): 6 * 16 * 2^-23 < 2^-16 of the
largest magnitude M that the sums are made of.  Where the result is 16 bits
and no state is asked for, products keep 16 bits instead of 24 (what
is left out is below 2^-16 of a product): 6 * 16 * 2^-16 / 2 < 2^-10 of M,
below the half step of M's own size.  M is the largest value of the
reference tensor, and for dg, which sums over the tokens of a chunk, the largest
such sum of |q||dq| + |k||dk|.  A decay floor or reset scales both sides alike."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import block_norm_np, gated_delta_np as onp
from selective_scan_ss2d_b200 import binding, build

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FINE, COARSE = 2.0 ** -16, 2.0 ** -10


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def make(B, L, HK, H, DK, DV, seed=0, decay=1.0):
    rng = np.random.default_rng([seed, B, L, H, DK, DV])
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)  # noqa: E731
    a = dict(q=unit(rng.standard_normal((B, L, HK, DK))), k=unit(rng.standard_normal((B, L, HK, DK))),
             v=rng.standard_normal((B, L, H, DV)))
    a["g"] = -decay * rng.uniform(0.0, 1.0, (B, L, H)) ** 3
    a["beta"] = rng.uniform(0.0, 1.0, (B, L, H))
    return a


# ------------------------------------------------------------------ oracle
def flat(a):
    return {n: v.reshape((-1,) + v.shape[2:]) for n, v in a.items()}


@pytest.mark.parametrize("reverse", [False, True])
def test_oracle_gradients_against_differences(reverse):
    a = flat(make(1, 7, 1, 2, 3, 2, seed=3))
    cu, rng = [0, 3, 3, 7], np.random.default_rng(1)
    h0, do, dh = rng.standard_normal((3, 2, 3, 2)), rng.standard_normal((7, 2, 2)), rng.standard_normal((3, 2, 3, 2))

    def loss(**x):
        y = {**a, "h0": h0, **x}
        o, h, _ = onp.forward(cu=cu, reverse=reverse, **y)
        return (o * do).sum() + (h * dh).sum()

    gr = onp.backward(cu=cu, do=do, h0=h0, dh_last=dh, reverse=reverse, **a)
    for n in ("q", "k", "v", "g", "beta", "h0"):
        x = h0 if n == "h0" else a[n]
        num, step = np.zeros_like(x), 1e-5
        for i in np.ndindex(x.shape):
            hi, lo = x.copy(), x.copy()
            hi[i] += step
            lo[i] -= step
            num[i] = (loss(**{n: hi}) - loss(**{n: lo})) / (2 * step)
        # truncation step^2 |f'''| / 6 and rounding 2^-53 |f| / step, both below 1e-8 at these sizes
        np.testing.assert_allclose(gr["d" + n], num, rtol=1e-6, atol=1e-7, err_msg=n)


def test_oracle_replaces_what_a_key_holds():
    """g = 0, |k| = 1, beta = 1: S^T k_t = v_t after every step, whatever was there."""
    a = flat(make(1, 9, 1, 1, 4, 3))
    a["g"][:], a["beta"][:] = 0.0, 1.0
    _, _, states = onp.forward(cu=[0, 9], **a)
    for t in range(9):
        np.testing.assert_allclose(states[0][t + 1][0].T @ a["k"][t, 0], a["v"][t, 0], atol=1e-12)


def test_oracle_orthonormal_keys_are_a_sum():
    """Keys that never meet: o_t = scale sum_j exp(sum of g after j) beta_j (q_t.k_j) v_j."""
    a = flat(make(1, 5, 1, 1, 5, 3))
    a["k"] = np.eye(5)[:, None, :]
    o, _, _ = onp.forward(cu=[0, 5], **a)
    c = np.cumsum(a["g"][:, 0])
    for t in range(5):
        want = sum(np.exp(c[t] - c[j]) * a["beta"][j, 0] * a["q"][t, 0, j] * a["v"][j, 0] for j in range(t + 1))
        np.testing.assert_allclose(o[t, 0], want * 5 ** -0.5, atol=1e-12)


# ---------------------------------------------------------------- refusals
def ptr():
    buf = (ctypes.c_float * 64)()
    addr = ctypes.addressof(buf)
    return buf, ctypes.c_void_p(addr + (-addr) % 16)


def _fwd(lib, p, nseq=1, L=8, HK=1, H=2, DK=16, DV=16, qs=16, ks=16, vs=32, dtype=1, nulls=(5, 7, 8)):
    a = [p] * 9
    for i in nulls:
        a[i] = None
    return lib.gated_delta_rule_fwd(*a, nseq, L, HK, H, DK, DV, qs, ks, vs, 1.0, 0, dtype, None)


def _bwd(lib, p, nseq=1, L=8, HK=1, H=2, DK=16, DV=16, qs=16, ks=16, vs=32, dtype=1, nulls=(5, 7, 13, 14)):
    a = [p] * 15
    for i in nulls:
        a[i] = None
    return lib.gated_delta_rule_bwd(*a, nseq, L, HK, H, DK, DV, qs, ks, vs, 1.0, 0, dtype, None)


def _step(lib, p, nseq=1, L=8, HK=1, H=2, DK=16, DV=16, qs=16, ks=16, vs=32, dtype=1, nulls=(6,)):
    a = [p] * 8
    for i in nulls:
        a[i] = None
    return lib.gated_delta_rule_step(*a, nseq, L, HK, H, DK, DV, qs, ks, vs, 1.0, dtype, None)


@pytest.mark.parametrize("call", [_fwd, _bwd, _step])
def test_argument_errors_are_reported_without_cuda(lib, call):
    keep, p = ptr()
    assert call(lib, p, nseq=-1) == -2
    assert call(lib, p, L=-1) == -2
    if call is not _step:
        assert call(lib, p, L=2 ** 31 - 1) == -2
    assert call(lib, p, HK=1, H=70000, vs=70000 * 16) == -2
    assert call(lib, p, dtype=5) == -3
    assert call(lib, p, HK=2, H=3, qs=32, ks=32, vs=48) == -14
    assert call(lib, p, HK=0, H=2) == -14
    for dk in (0, 8, 24, 144):
        assert call(lib, p, DK=dk, qs=200, ks=200) == -14
    for dv in (0, 8, 100, 272):
        assert call(lib, p, DV=dv, vs=600) == -14
    assert call(lib, p, qs=15) == -13
    assert call(lib, p, ks=8) == -13
    assert call(lib, p, vs=31) == -13
    assert call(lib, p, qs=20) == -6            # rows off the 16-byte boundaries
    assert call(lib, p, nulls=(0,)) == -1
    assert call(lib, p, nulls=(4,)) == -1
    assert call(lib, ctypes.c_void_p(p.value + 4)) == -6
    assert call(lib, p, nseq=0, nulls=range(8)) == 0
    assert binding.ss2d_status_string(-14) != "unknown status"


def test_more_refusals(lib):
    keep, p = ptr()
    assert _fwd(lib, p, L=0, nulls=range(9)) == 0
    assert _bwd(lib, p, L=0, nulls=range(15)) == 0
    assert _bwd(lib, p, nulls=(6,)) == -1
    assert _bwd(lib, p, nulls=(12,)) == -1
    assert _step(lib, p, nseq=9, L=8, nulls=(6,)) == -2   # fewer states than rows, no slots


def test_binding_validates_tensors(lib):
    q, v, g = torch.zeros(1, 4, 1, 16), torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="device tensors only"):
        binding.gated_delta_rule_fwd(q, q, v, g, g)
    with pytest.raises(ValueError, match="inconsistent"):
        binding.gated_delta_rule_fwd(q, q[:, :3], v, g, g)
    with pytest.raises(ValueError, match="inconsistent"):
        binding.gated_delta_rule_bwd(q, q, v, g[..., :1], g, v)
    with pytest.raises(TypeError):
        binding.gated_delta_rule_fwd(q.double(), q, v, g, g)
    with pytest.raises(TypeError):
        binding.gated_delta_rule_fwd(q, q.half(), v, g, g)
    with pytest.raises(TypeError):
        binding.gated_delta_rule_step(q[0], q[0], v[0], g[0].half(), g[0], torch.zeros(4, 2, 16, 16))


def test_token_strides(lib):
    w = torch.zeros(3, 5, 100)
    assert binding._token_stride(w[..., :32].unflatten(-1, (2, 16)), "q") == 100
    assert binding._token_stride(w[:1, :, :32].unflatten(-1, (2, 16)), "q") == 100
    assert binding._token_stride(w[:, :1, :32].unflatten(-1, (2, 16)), "q") == 500
    assert binding._token_stride(w[0, :, 4:36].unflatten(-1, (2, 16)), "q") == 100
    assert binding._token_stride(torch.zeros(2, 3, 2, 16), "q") == 32
    for bad in (w[:, :4, :32].unflatten(-1, (2, 16)), w[..., :64:2].unflatten(-1, (2, 16)),
                w[..., :32].unflatten(-1, (16, 2)).transpose(-1, -2), torch.zeros(1, 1, 2, 16).expand(3, 4, 2, 16)):
        with pytest.raises(ValueError, match="one stride"):
            binding._token_stride(bad, "q")


# --------------------------------------------------------------------- GPU
def dev(a, dtype):
    t = {n: torch.from_numpy(np.ascontiguousarray(v)).to(DT[dtype] if n in "qkv" else torch.float32).cuda()
         for n, v in a.items()}
    return t, {n: v.double().cpu().numpy().reshape((-1,) + tuple(v.shape[2:])) for n, v in t.items()}


def near(got, ref, dt, tol, M, what):
    got = got.double().cpu().numpy().reshape(ref.shape)
    half = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    bound = half * np.maximum(np.abs(ref), torch.finfo(dt).tiny) + tol * M
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.2f} of the bound at " \
        f"{np.unravel_index(np.argmax(err / bound), err.shape)}"


def mag(*a):
    return max([1e-30] + [float(np.abs(x).max()) for x in a if x is not None and x.size])


def run_fwd(a, dtype, cu=None, state=True, reverse=False, scale=None, seed=0, wrap=None):
    t, f = dev(a, dtype)
    B, L = a["q"].shape[:2]
    H, DK, DV = a["v"].shape[2], a["q"].shape[3], a["v"].shape[3]
    bounds = [L * b for b in range(B + 1)] if cu is None else cu
    nseq = len(bounds) - 1
    rng = np.random.default_rng(seed + 100)
    h0 = torch.from_numpy(rng.standard_normal((nseq, H, DK, DV)) * 0.5).float().cuda() if state else None
    cut = torch.tensor(cu, dtype=torch.int32).cuda() if cu is not None else None
    if wrap:
        t = wrap(t)
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, cu_seqlens=cut, reverse=reverse, final_state=state, scale=scale)
    torch.cuda.synchronize()
    fh = h0.double().cpu().numpy() if state else None
    ro, rh, _ = onp.forward(**f, cu=bounds, h0=fh, scale=scale, reverse=reverse)
    inside = np.zeros(B * L, bool)
    for n in range(nseq):
        inside[bounds[n]:bounds[n + 1]] = True
    tol = FINE if state or dtype == "f32" else COARSE
    # o is made of q.S and of v: their sizes
    sc = DK ** -0.5 if scale is None else abs(scale)
    M = mag(ro, sc * f["v"] * mag(f["q"]))
    got = o.flatten(0, 1)[torch.from_numpy(inside).cuda()]
    near(got, ro[inside], DT[dtype], tol, M, "o")
    if state:
        near(h, rh, torch.float32, FINE, mag(rh, f["v"] * mag(f["k"])), "h_last")
    else:
        assert h is None
    return t, f, h0, cut, bounds, o, h


def run_bwd(a, dtype, cu=None, state=True, reverse=False, scale=None, seed=0, wrap=None):
    t, f, h0, cut, bounds, o, h = run_fwd(a, dtype, cu, state, reverse, scale, seed, wrap)
    rng = np.random.default_rng(seed + 200)
    do = torch.from_numpy(rng.standard_normal(a["v"].shape)).to(DT[dtype]).cuda()
    dh = torch.from_numpy(rng.standard_normal(tuple(h.shape)) * 0.5).float().cuda() if state else None
    g = binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=dh, cu_seqlens=cut, reverse=reverse, scale=scale)
    torch.cuda.synchronize()
    n64 = lambda x: None if x is None else x.double().cpu().numpy()  # noqa: E731
    fdo = n64(do).reshape(f["v"].shape)
    ref = onp.backward(**f, cu=bounds, do=fdo, h0=n64(h0), dh_last=n64(dh), scale=scale, reverse=reverse)
    for n in ("dq", "dk", "dv"):
        near(g[n], ref[n], DT[dtype], FINE if dtype == "f32" else COARSE / 2, mag(ref[n]), n)
    near(g["dbeta"], ref["dbeta"], torch.float32, FINE, mag(ref["dbeta"], ref["dv"] * mag(f["v"])), "dbeta")
    dot = (np.abs(f["q"]) * np.abs(ref["dq"])).sum(-1).max(1) + (np.abs(f["k"]) * np.abs(ref["dk"])).sum(-1).max(1)
    near(g["dg"], ref["dg"], torch.float32, FINE, max(mag(ref["dg"]), max(
        float(dot[i:i + 64].sum()) for i in range(0, len(dot), 32))), "dg")
    if state:
        near(g["dh0"], ref["dh0"], torch.float32, FINE, mag(ref["dh0"], fdo), "dh0")
    else:
        assert g["dh0"] is None
    return t, g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("L", [1, 2, 4, 5, 63, 64, 65, 130])
def test_forward_lengths(L, dtype):
    a = make(2, L, 1, 2, 32, 48, seed=L)
    run_fwd(a, dtype)
    run_fwd(a, dtype, state=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("HK,H,DK,DV", [(1, 1, 16, 16), (2, 2, 64, 64), (1, 3, 48, 80), (2, 4, 128, 128),
                                        (1, 1, 96, 192), (1, 2, 128, 256), (3, 3, 64, 112)])
def test_forward_head_layouts(HK, H, DK, DV, dtype):
    run_fwd(make(1, 100, HK, H, DK, DV), dtype)
    run_fwd(make(2, 70, HK, H, DK, DV), dtype, state=False, reverse=True, scale=0.7)


@pytest.mark.gpu
def test_forward_many_wide_heads():
    """enough heads for eight warps a CTA"""
    run_fwd(make(2, 70, 40, 80, 64, 128), "bf16")
    run_fwd(make(2, 66, 40, 80, 128, 96), "f16", state=False)


CUTS = [[0, 70], [0, 0, 64, 64, 130, 131, 200], [5, 9, 9, 140, 203], [0, 0, 0], [199, 203]]


@pytest.mark.gpu
@pytest.mark.parametrize("cu", CUTS)
@pytest.mark.parametrize("dtype,reverse", [("bf16", False), ("f16", True), ("f32", False)])
def test_packed_sequences(cu, dtype, reverse):
    a = make(1, 207, 1, 2, 32, 32)
    run_bwd(a, dtype, cu=cu, reverse=reverse)
    run_fwd(a, dtype, cu=cu, reverse=not reverse, state=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("L", [1, 3, 64, 65, 129])
def test_backward_lengths(L, dtype):
    run_bwd(make(2, L, 1, 2, 32, 48, seed=L), dtype)
    run_bwd(make(1, L, 2, 2, 64, 16, seed=L), dtype, state=False, reverse=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("HK,H,DK,DV", [(1, 1, 16, 16), (2, 2, 64, 64), (1, 3, 48, 80), (2, 4, 128, 128),
                                        (1, 1, 96, 192), (1, 2, 128, 256)])
def test_backward_head_layouts(HK, H, DK, DV, dtype):
    run_bwd(make(1, 100, HK, H, DK, DV), dtype, scale=0.5)


@pytest.mark.gpu
def test_backward_many_wide_heads():
    run_bwd(make(2, 70, 40, 80, 64, 128), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.0, 30.0])
def test_long_chain_and_strong_decay(dtype, decay):
    run_bwd(make(1, 700, 1, 1, 64, 64, decay=decay), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,DK,DV,L", [("bf16", 32, 48, 2100), ("f32", 64, 16, 2048), ("f16", 128, 80, 2050),
                                           ("bf16", 96, 128, 2600)])
def test_long_chains_in_segments(dtype, DK, DV, L):
    """few heads and long sequences: the chain is cut, its segments run from the states that lead to them"""
    run_bwd(make(1, L, 1, 1, DK, DV, decay=0.3), dtype)
    run_fwd(make(1, L, 1, 1, DK, DV, decay=0.0), dtype, state=False, reverse=True)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 0, 6500, 6501, 6990], [3, 2900, 2900, 6980, 6990], [0, 64, 640, 6000, 6990]])
@pytest.mark.parametrize("dtype,reverse", [("bf16", False), ("f32", True)])
def test_packed_long_chains_in_segments(cu, dtype, reverse):
    run_bwd(make(1, 7001, 1, 2, 32, 32, decay=0.2), dtype, cu=cu, reverse=reverse)


@pytest.mark.gpu
def test_resets_by_infinite_decay():
    """g = -inf and the lowest float forget the state: the same as a sequence that starts there"""
    a = make(1, 150, 1, 2, 32, 32)
    t, _ = dev(a, "bf16")
    whole, _ = binding.gated_delta_rule_fwd(**t, final_state=True)
    t["g"][0, 40] = -np.inf
    t["g"][0, 100] = torch.finfo(torch.float32).min
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    cu = torch.tensor([0, 40, 100, 150], dtype=torch.int32).cuda()
    t["g"][0, 40] = t["g"][0, 100] = 0.0
    o2, h2 = binding.gated_delta_rule_fwd(**t, cu_seqlens=cu, final_state=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:, :40], whole[:, :40])
    # the same sums split at other tokens: float32 rounding, then the store's half step on both sides; a bfloat16 has
    # 8 significant bits, so a half step is up to 2^-8 of the value, and two of them 2^-7
    far = (o.float() - o2.float()).abs() - 2 ** -7 * o2.float().abs() - FINE * o2.float().abs().max()
    assert float(far.max()) <= 0
    far = (h[0] - h2[2]).abs() - FINE * h2.abs().max()
    assert float(far.max()) <= 0
    t["g"][0, 40] = -np.inf
    gr = binding.gated_delta_rule_bwd(**t, do=o)
    torch.cuda.synchronize()
    assert all(torch.isfinite(v).all() for v in gr.values() if v is not None)
    # exactly zero, as a sum of terms that cancel: each is off by FINE of the largest like any dg
    assert float(gr["dg"][0, 40].abs().max()) <= FINE * float(gr["dg"].abs().max())


@pytest.mark.gpu
def test_rows_outside_every_sequence_are_left_alone():
    a = make(1, 150, 1, 2, 32, 32)
    t, _ = dev(a, "bf16")
    for n in t:   # what nobody reads may hold anything
        t[n][0, 120:] = float("nan")
        t[n][0, :7] = float("inf")
    cu = torch.tensor([7, 60, 120], dtype=torch.int32).cuda()
    o = torch.full((1, 150, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    binding.gated_delta_rule_fwd(**t, cu_seqlens=cu, o=o)
    g = binding.gated_delta_rule_bwd(**t, do=torch.ones_like(o), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.all(o[0, 120:] == 3) and torch.all(o[0, :7] == 3) and torch.isfinite(o).all()
    for n, v in g.items():
        if v is not None:
            assert torch.isfinite(v).all() and not v[0, 120:].any() and not v[0, :7].any(), n


@pytest.mark.gpu
def test_positions_outside_the_tokens_are_moved_inside():
    a = make(1, 100, 1, 1, 16, 16)
    t, _ = dev(a, "bf16")
    big = torch.tensor([-5, 40, 2 ** 31 - 1], dtype=torch.int32).cuda()
    ok = torch.tensor([0, 40, 100], dtype=torch.int32).cuda()
    assert torch.equal(binding.gated_delta_rule_fwd(**t, cu_seqlens=big)[0],
                       binding.gated_delta_rule_fwd(**t, cu_seqlens=ok)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_of_one_projection(dtype):
    def wrap(t):
        qkv = torch.cat([t[n].flatten(2) for n in "qkv"] + [t["v"].flatten(2)[..., :16]], -1)
        out, at = dict(t), 0
        for n in "qkv":
            w = t[n].shape[2] * t[n].shape[3]
            out[n] = qkv[..., at:at + w].unflatten(-1, t[n].shape[2:])
            at += w
        assert not out["q"].is_contiguous()
        return out

    run_bwd(make(2, 75, 2, 4, 32, 48), dtype, wrap=wrap)
    run_fwd(make(3, 3, 2, 4, 32, 48), dtype, wrap=wrap)


@pytest.mark.gpu
def test_split_sequence_continues_from_its_state():
    a = make(1, 210, 1, 2, 64, 64)
    t, _ = dev(a, "bf16")
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    o1, h1 = binding.gated_delta_rule_fwd(**{n: v[:, :128].contiguous() for n, v in t.items()}, final_state=True)
    o2, h2 = binding.gated_delta_rule_fwd(**{n: v[:, 128:].contiguous() for n, v in t.items()}, h0=h1, h_last=h1)
    torch.cuda.synchronize()
    assert h2.data_ptr() == h1.data_ptr()
    assert torch.equal(o, torch.cat([o1, o2], 1)) and torch.equal(h, h2)   # a whole number of chunks


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,HK,H,DK,DV", [(1, 1, 1, 16, 16), (3, 2, 4, 64, 64), (5, 1, 3, 48, 80), (2, 1, 2, 128, 256),
                                          (70, 2, 2, 128, 128), (4, 3, 3, 96, 192)])
def test_step(B, HK, H, DK, DV, dtype):
    a = make(B, 1, HK, H, DK, DV)
    t, f = dev(a, dtype)
    s = {n: v[:, 0].contiguous() for n, v in t.items()}
    rng = np.random.default_rng(B)
    pool = torch.from_numpy(rng.standard_normal((2 * B + 1, H, DK, DV))).float().cuda()
    slots = torch.from_numpy(rng.permutation(2 * B + 1)[:B].astype(np.int32)).cuda()
    if B > 2:
        slots[1] = -1
    before = pool.clone()
    o = binding.gated_delta_rule_step(**s, state=pool, slots=slots)
    torch.cuda.synchronize()
    idx = slots.long().cpu().numpy()
    live = idx >= 0
    h0 = before.double().cpu().numpy()[np.where(live, idx, 0)]
    ro, rh, _ = onp.forward(**f, cu=list(range(B + 1)), h0=h0)
    near(o[torch.from_numpy(live).cuda()], ro[live], DT[dtype], FINE, mag(ro), "o")
    assert not o[torch.from_numpy(~live).cuda()].any()
    near(pool[slots.long()[torch.from_numpy(live).cuda()]], rh[live], torch.float32, FINE, mag(rh), "state")
    rest = np.setdiff1d(np.arange(2 * B + 1), idx[live])
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.gpu
def test_step_slots_outside_and_named_twice():
    a = make(5, 1, 1, 2, 32, 32)
    t, _ = dev(a, "bf16")
    s = {n: v[:, 0].contiguous() for n, v in t.items()}
    pool = torch.ones(4, 2, 32, 32, device="cuda")
    one = pool.clone()
    slots = torch.tensor([2, 7, 2, -3, 0], dtype=torch.int32).cuda()
    o = binding.gated_delta_rule_step(**s, state=pool, slots=slots)
    o1 = binding.gated_delta_rule_step(**{n: v[[0, 4]].contiguous() for n, v in s.items()}, state=one,
                                       slots=slots[[0, 4]].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(pool, one) and torch.equal(o[[0, 4]], o1) and not o[1:4].any()
    none = torch.empty(0, 2, 32, 32, device="cuda")
    assert not binding.gated_delta_rule_step(**s, state=none, slots=slots).any()


@pytest.mark.gpu
def test_steps_follow_the_chunked_pass():
    """tokens one at a time, the states in place, give the sequence's outputs and state"""
    a = make(2, 70, 1, 2, 64, 32)
    t, _ = dev(a, "f32")
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    pool = torch.zeros_like(h)
    outs = []
    for i in range(70):
        outs.append(binding.gated_delta_rule_step(**{n: v[:, i].contiguous() for n, v in t.items()}, state=pool))
    torch.cuda.synchronize()
    # 70 steps of float32 rounding against the chunks': both within FINE of the exact values
    assert float((torch.stack(outs, 1) - o).abs().max()) <= 2 * FINE * float(o.abs().max())
    assert float((pool - h).abs().max()) <= 2 * FINE * float(h.abs().max())


@pytest.mark.gpu
def test_repeatable_streams_and_graphs():
    a = make(1, 300, 2, 4, 64, 64)
    t, _ = dev(a, "bf16")
    h0 = torch.ones(1, 4, 64, 64, device="cuda") * 0.1
    do = torch.ones_like(t["v"])
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, final_state=True)
    g = binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(2):   # two calls at once, twice
        for s in streams:
            with torch.cuda.stream(s):
                o1, h1 = binding.gated_delta_rule_fwd(**t, h0=h0, final_state=True)
                got.append((o1, h1, binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=h)))
    torch.cuda.synchronize()
    for o1, h1, g1 in got:
        assert torch.equal(o, o1) and torch.equal(h, h1) and all(torch.equal(g[n], g1[n]) for n in g)
    graphs, keep = [], []
    v = t["v"].clone()
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o2, h2 = binding.gated_delta_rule_fwd(**{**t, "v": v}, h0=h0, final_state=True)
            g2 = binding.gated_delta_rule_bwd(**{**t, "v": v}, do=do, h0=h0, dh_last=h2)
        graphs.append(gr)
        keep.append((o2, h2, g2))
    for f in (1.0, -2.0):
        v.copy_(t["v"] * f)
        for i, s in enumerate(streams):   # both graphs at once
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        o3, h3 = binding.gated_delta_rule_fwd(**{**t, "v": v}, h0=h0, final_state=True)
        g3 = binding.gated_delta_rule_bwd(**{**t, "v": v}, do=do, h0=h0, dh_last=h3)
        for o2, h2, g2 in keep:
            assert torch.equal(o2, o3) and torch.equal(h2, h3) and all(torch.equal(g2[n], g3[n]) for n in g2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_channels_of_very_different_size(dtype):
    """every value channel is a recurrence of its own: scaled by a power of two, it keeps its bits"""
    a = make(2, 150, 1, 2, 64, 48)
    t, _ = dev(dict(a, v=a["v"] / 64), dtype)
    up = 2.0 ** (torch.arange(48) % 17).cuda()   # values of about 2^-6 .. 2^10, the same bits as the stored ones
    u = dict(t, v=(t["v"].float() * up).to(t["v"].dtype))
    assert torch.equal(t["v"].float() * up, u["v"].float())
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    o1, h1 = binding.gated_delta_rule_fwd(**u, final_state=True)
    assert torch.equal(h * up[:, None].T, h1)
    # float16 outputs below 2^-14 are rounded to multiples of 2^-24 before they are scaled here
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    assert bool(((o.float() * up - o1.float()).abs() <= tiny * up).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_no_tokens_and_no_sequences(dtype):
    """states pass through sequences of nothing; tokens without sequences have no gradient"""
    def call(L):
        new = lambda *s: torch.ones(*s, dtype=DT[dtype], device="cuda")  # noqa: E731
        g = torch.ones(1, L, 2, device="cuda")
        return dict(q=new(1, L, 2, 16), k=new(1, L, 2, 16), v=new(1, L, 2, 32), g=g, beta=g)

    h0 = torch.rand(3, 2, 16, 32, device="cuda")
    t, cu = call(0), torch.zeros(4, dtype=torch.int32, device="cuda")
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, cu_seqlens=cu, final_state=True)
    gr = binding.gated_delta_rule_bwd(**t, do=t["v"], h0=h0, dh_last=2 * h0, cu_seqlens=cu)
    assert o.shape == t["v"].shape and torch.equal(h, h0) and torch.equal(gr["dh0"], 2 * h0)
    t = call(70)
    gr = binding.gated_delta_rule_bwd(**t, do=t["v"], cu_seqlens=cu[:1])
    assert not any(gr[n].any() for n in ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_another_stream_than_the_current_one(raw):
    """everything that a call writes, rows of no sequence among it, is written on its stream"""
    t, _ = dev(make(1, 150, 1, 2, 32, 32), "bf16")
    do = torch.ones_like(t["v"])
    cu = torch.tensor([7, 60, 120], dtype=torch.int32).cuda()
    want = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)   # the current stream is behind for some 25 ms
    got = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu, stream=s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    assert all(got[n] is None or torch.equal(got[n], want[n]) for n in want)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """tokens 2^24 values apart, and a state that begins past 2^31 values of the pool: the bits of packed ones"""
    t, _ = dev(make(1, 135, 1, 1, 16, 32), "bf16")
    do = torch.ones_like(t["v"])
    far = torch.empty(135, 1, 1 << 24, dtype=torch.bfloat16, device="cuda")
    wide = dict(t)
    for n, at, w in (("q", 0, 16), ("k", 16, 16), ("v", 32, 32)):
        wide[n] = far[None, :, :, at:at + w]
        wide[n].copy_(t[n])
    assert wide["v"].stride(1) * 134 > 2 ** 31
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    o1, h1 = binding.gated_delta_rule_fwd(**wide, final_state=True)
    g, g1 = (binding.gated_delta_rule_bwd(**u, do=do) for u in (t, wide))
    assert torch.equal(o, o1) and torch.equal(h, h1)
    assert all(g[n] is None or torch.equal(g[n], g1[n]) for n in g)
    del far, wide
    n = (1 << 31) // (16 * 32) + 2
    pool = torch.empty(n, 1, 16, 32, device="cuda")
    small = torch.ones(2, 1, 16, 32, device="cuda")
    pool[-2:] = 1
    one = {k: v[0, :2] for k, v in t.items()}
    slots = torch.tensor([n - 1, n - 2], dtype=torch.int32).cuda()
    o2 = binding.gated_delta_rule_step(**one, state=pool, slots=slots)
    o3 = binding.gated_delta_rule_step(**one, state=small, slots=torch.tensor([1, 0], dtype=torch.int32).cuda())
    assert torch.equal(o2, o3) and torch.equal(pool[-2:], small)


@pytest.mark.gpu
def test_a_block_of_them_together():
    """Pre-norm -> q, k normalised by the block norm -> delta rule -> gated norm -> residual + next norm, and back,
    against the oracles' chain in float64 (float32 inputs, so that only float32 rounding is between them)."""
    B, L, H, D = 2, 90, 2, 32
    rng = np.random.default_rng(7)
    f = {n: rng.standard_normal((B, L, H, D)) for n in ("q", "k", "v", "z")}
    r = rng.standard_normal((B, L, H * D))
    a = make(B, L, H, H, D, D)
    w, wr = 1 + 0.1 * rng.standard_normal(D), 1 + 0.1 * rng.standard_normal(H * D)
    unit = np.full(D, D ** -0.5)   # an rms norm with this weight has length 1
    dev32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).float().cuda()  # noqa: E731
    t = {n: dev32(x) for n, x in f.items()}
    t64 = {n: x.double().cpu().numpy() for n, x in t.items()}
    tw, twr, tu, tr, tg, tb = map(dev32, (w, wr, unit, r, a["g"], a["beta"]))
    qn = binding.block_norm_fwd(t["q"], post="rms", w_post=tu, eps=0.0)[0]
    kn = binding.block_norm_fwd(t["k"], post="rms", w_post=tu, eps=0.0)[0]
    o, _ = binding.gated_delta_rule_fwd(qn, kn, t["v"], tg, tb)
    on = binding.block_norm_fwd(o, z=t["z"], post="rms", w_post=tw)[0]
    r1, y = binding.block_norm_fwd(on.flatten(2), r=tr, pre="layer", w_pre=twr)
    dy = dev32(rng.standard_normal(r.shape))
    g1 = binding.block_norm_bwd(on.flatten(2), None, dy, r_out=r1, pre="layer", w_pre=twr)
    g2 = binding.block_norm_bwd(o, g1["dx"].view_as(o), z=t["z"], post="rms", w_post=tw, residual=False)
    g3 = binding.gated_delta_rule_bwd(qn, kn, t["v"], tg, tb, g2["dx"])
    g4 = binding.block_norm_bwd(t["q"], g3["dq"], post="rms", w_post=tu, eps=0.0, residual=False)
    torch.cuda.synchronize()
    n64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    N = block_norm_np
    eq, _ = N.block_norm_fwd(t64["q"], post="rms", w_post=n64(tu), eps=0.0)
    ek, _ = N.block_norm_fwd(t64["k"], post="rms", w_post=n64(tu), eps=0.0)
    fl = lambda x: x.reshape((-1,) + x.shape[2:])  # noqa: E731
    cu = [0, L, 2 * L]
    eo = onp.forward(fl(eq), fl(ek), fl(t64["v"]), fl(n64(tg)), fl(n64(tb)), cu)[0].reshape(f["v"].shape)
    en, _ = N.block_norm_fwd(eo, z=t64["z"], post="rms", w_post=n64(tw))
    er, ey = N.block_norm_fwd(en.reshape(r.shape), r=n64(tr), pre="layer", w_pre=n64(twr))
    e1 = N.block_norm_bwd(en.reshape(r.shape), None, n64(dy), r_out=er, pre="layer", w_pre=n64(twr))
    e2 = N.block_norm_bwd(eo, e1["dx"].reshape(eo.shape), z=t64["z"], post="rms", w_post=n64(tw))
    e3 = onp.backward(fl(eq), fl(ek), fl(t64["v"]), fl(n64(tg)), fl(n64(tb)), cu, fl(e2["dx"]))
    e4 = N.block_norm_bwd(t64["q"], e3["dq"].reshape(eq.shape), post="rms", w_post=n64(tu), eps=0.0)
    # a norm divides by its row's size: errors of FINE of the largest value grow by (largest / smallest row) twice
    big = float(np.sqrt((eo ** 2).mean(-1)).max() / np.sqrt((eo ** 2).mean(-1)).min())
    for what, got, ref, amp in (("o", o, eo, 1), ("y", y, ey, big), ("dz", g2["dz"], e2["dz"], big * big),
                                ("dx", g2["dx"], e2["dx"], big * big), ("dv", g3["dv"], e3["dv"], big * big),
                                ("dg", g3["dg"], e3["dg"], 64 * big * big), ("dq", g4["dx"], e4["dx"], big * big)):
        near(got, ref, torch.float32, FINE * amp, mag(ref), what)
