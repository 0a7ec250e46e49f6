"""The gated delta rule at the edges of what its calls allow: the default
stream by its handle, rows of no sequence in a new output, no value heads; and
how far off it is as a whole, in every form of the chain and for many of them.

What is kept in float32 is off by less than WHOLE of its L2 norm.  A product of
three-part operands truncates once at its full size (2^-23, the small parts are summed
first) and is joined by rounding additions, up to eight to a sum, whose errors of
2^-24 add like sqrt(8); a result is at most six such sums in a row, none of which
lets an error grow (|k| <= 1, beta <= 1, g <= 0): 6 * (2^-23 + sqrt(8) * 2^-24) = 1.7e-6 <
2^-19.  Two scaled float16 parts hold 2^-23 of a column's largest value, four times
its root mean square: 2^-21 / sqrt(3) for each of the six, below 2^-19 as well.  Two bf16
parts, or parts summed where the whole sum truncates each of them, do not reach it."""
from __future__ import annotations

import ctypes
import threading

import numpy as np
import pytest
import torch

import test_gated_delta as td
from oracle import gated_delta_np as onp
from selective_scan_ss2d_b200 import binding

WHOLE = 2.0 ** -19

lib = td.lib   # the fixture: the built library


def test_backward_without_value_heads_is_refused(lib):
    """nothing would write dq and dk"""
    keep, p = td.ptr()
    assert td._bwd(lib, p, HK=1, H=0, vs=0) == -14
    assert td._bwd(lib, p, HK=0, H=0, qs=0, ks=0, vs=0) == 0
    assert td._fwd(lib, p, HK=1, H=0, vs=0) == 0   # an output of no heads


def test_alignment_of_values_read_one_by_one(lib):
    """g, beta, positions and slots may start at any value; half of one is refused"""
    keep, p = td.ptr()
    at = lambda n: ctypes.c_void_p(p.value + n)  # noqa: E731
    head = (1, 8, 1, 2, 16, 16, 16, 16, 32, 1.0)
    for off, want in ((4, -9), (2, -6)):   # host memory, once the alignment is in order
        for i in (3, 4, 8):
            a = [p, p, p, p, p, None, p, None, None]
            a[i] = at(off)
            assert lib.gated_delta_rule_fwd(*a, *head, 0, 1, None) in ((want, -8) if want == -9 else (want,)), (off, i)
        for i in (3, 4, 11, 12, 14):
            a = [p] * 5 + [None, p, None] + [p] * 5 + [None, None]
            a[i] = at(off)
            assert lib.gated_delta_rule_bwd(*a, *head, 0, 1, None) in ((want, -8) if want == -9 else (want,)), (off, i)
        for i in (3, 4, 6):
            a = [p] * 6 + [None, p]
            a[i] = at(off)
            assert lib.gated_delta_rule_step(*a, 1, 8, *head[2:], 1, None) in ((want, -8) if want == -9 else (want,)), (off, i)
    for i in (0, 1, 2, 6):
        a = [p, p, p, p, p, None, p, None, None]
        a[i] = at(4)
        assert lib.gated_delta_rule_fwd(*a, *head, 0, 1, None) == -6, i


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 3])
def test_tokens_of_one_sequence_one_by_one(H):
    """g[:, t] and beta[:, t] of a batch of one, as they lie in the sequence's tensors"""
    t, _ = td.dev(td.make(1, 9, 1, H, 32, 16), "bf16")
    pool = torch.zeros(2, 1, H, 32, 16, device="cuda")
    for i in range(9):
        row = {n: v[:, i] for n, v in t.items()}
        o = binding.gated_delta_rule_step(**row, state=pool[0])
        o1 = binding.gated_delta_rule_step(**{n: v.clone() for n, v in row.items()}, state=pool[1])
        assert torch.equal(o, o1)
    assert torch.equal(pool[0], pool[1]) and pool.any()
    far = {n: torch.cat([v[:, :1], v], 1)[:, 1:] for n, v in t.items()}   # from the second row of a batch of one on
    cu = torch.tensor([9, 0, 4, 9], dtype=torch.int32).cuda()[1:]
    do = torch.ones_like(t["v"])
    for fn, kw in ((binding.gated_delta_rule_fwd, {}), (binding.gated_delta_rule_bwd, dict(do=do))):
        a, b = fn(**far, **kw, cu_seqlens=cu), fn(**t, **kw, cu_seqlens=cu.clone())
        a, b = (x.values() if isinstance(x, dict) else x for x in (a, b))
        assert all(x is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_default_stream_by_its_handle():
    """stream = 0 is the default stream, for a call's kernels and for the zeros of rows in no sequence"""
    t, _ = td.dev(td.make(1, 150, 1, 2, 32, 32), "bf16")
    do = torch.ones_like(t["v"])
    cu = torch.tensor([7, 60, 120], dtype=torch.int32).cuda()
    assert torch.cuda.default_stream().cuda_stream == 0
    want = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu)
    busy = [torch.cuda.Stream() for _ in range(64)]   # whatever other stream a call would use is behind
    torch.cuda.synchronize()
    for s in busy:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    got = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu, stream=0)
    torch.cuda.synchronize()
    assert all(got[n] is None or torch.equal(got[n], want[n]) for n in want)


@pytest.mark.gpu
@pytest.mark.parametrize("L,cu", [(150, [7, 60, 120]), (150, [0, 149]), (150, [3]), (4, [1, 2]), (70, [70, 70])])
def test_rows_of_no_sequence_are_zero_in_a_new_output(L, cu):
    t, _ = td.dev(td.make(1, L, 1, 2, 32, 32), "bf16")
    for _ in range(4):   # what the allocator hands out next holds NaN
        torch.full_like(t["v"], float("nan"))
    o, _ = binding.gated_delta_rule_fwd(**t, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert not o[0, :cu[0]].any() and not o[0, cu[-1]:].any()
    assert bool(o[0, cu[0]:cu[-1]].any()) == (cu[-1] > cu[0])


def whole(got, ref, what, of=None):
    """off by WHOLE of the reference's L2 norm (or of `of`'s, whose sum the reference is)"""
    n = float(np.linalg.norm(ref if of is None else np.maximum(np.abs(ref), of)))
    err = float(np.linalg.norm(got.double().cpu().numpy().reshape(ref.shape) - ref))
    assert err <= WHOLE * n, f"{what}: {err / n:.2e}"


def run(a, dtype, cu=None, reverse=False):
    """forward, backward, and forward without states, against the oracle sequence by sequence"""
    t, f = td.dev(a, dtype)
    B, L, HK, DK = a["q"].shape
    H, DV = a["v"].shape[2:]
    bounds = [L * b for b in range(B + 1)] if cu is None else list(cu)
    nseq = len(bounds) - 1
    rng = np.random.default_rng([nseq, L, H])
    new = lambda dt, *s: torch.from_numpy(rng.standard_normal(s)).to(dt).cuda()  # noqa: E731
    h0, dh = 0.5 * new(torch.float32, nseq, H, DK, DV), 0.5 * new(torch.float32, nseq, H, DK, DV)
    do = new(td.DT[dtype], B, L, H, DV)
    kw = dict(cu_seqlens=None if cu is None else torch.tensor(bounds, dtype=torch.int32).cuda(), reverse=reverse)
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, final_state=True, **kw)
    g = binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=dh, **kw)
    o2, none = binding.gated_delta_rule_fwd(**t, h0=h0, **kw)
    torch.cuda.synchronize()
    n64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    fh, fdh, fdo = n64(h0), n64(dh), n64(do).reshape(f["v"].shape)
    ref = {n: np.zeros_like(f[m]) for n, m in (("o", "v"), ("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"),
                                               ("dbeta", "g"))}
    ref["h"], ref["dh0"] = np.zeros_like(fh), np.zeros_like(fh)
    amp = np.zeros(f["g"].shape)   # what dg is a sum of: |q||dq| + |k||dk| from a token to its chunk's end
    for n in range(nseq):
        at = slice(bounds[n], bounds[n + 1])
        x, one = {m: v[at] for m, v in f.items()}, [0, bounds[n + 1] - bounds[n]]
        ref["o"][at], rh, _ = onp.forward(**x, cu=one, h0=fh[n:n + 1], reverse=reverse)
        ref["h"][n] = rh[0]
        r = onp.backward(**x, cu=one, do=fdo[at], h0=fh[n:n + 1], dh_last=fdh[n:n + 1], reverse=reverse)
        for m in ("dq", "dk", "dv", "dg", "dbeta"):
            ref[m][at] = r[m]
        ref["dh0"][n] = r["dh0"][0]
        dot = sum(np.abs(x[m] * r["d" + m]).sum(-1).repeat(H // HK, 1) for m in "qk")
        dot = dot[::-1] if reverse else dot   # in the order of reading
        sums = np.concatenate([dot[i:i + 64][::-1].cumsum(0)[::-1] for i in range(0, len(dot), 64)] or [dot])
        amp[at] = sums[::-1] if reverse else sums
    names = [("h", h, None), ("dg", g["dg"], amp), ("dbeta", g["dbeta"], None), ("dh0", g["dh0"], None)]
    if dtype == "f32":
        names += [("o", o, None)] + [(m, g[m], None) for m in ("dq", "dk", "dv")]
    for m, got, of in names:
        whole(got, ref[m], m, of)
    # 16-bit outputs: their rounding, and by element
    M = td.mag(ref["o"], f["v"])
    td.near(o, ref["o"], td.DT[dtype], td.FINE, M, "o")
    assert none is None
    td.near(o2, ref["o"], td.DT[dtype], td.FINE if dtype == "f32" else td.COARSE, M, "o without states")
    for m in ("dq", "dk", "dv"):
        td.near(g[m], ref[m], td.DT[dtype], td.FINE if dtype == "f32" else td.COARSE / 2, td.mag(ref[m]), m)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("HK,H,DK,DV,L", [(1, 2, 64, 64, 200), (1, 2, 128, 128, 200), (2, 2, 48, 80, 130),
                                          (1, 1, 64, 48, 2100), (1, 1, 128, 64, 2090)])
def test_float32_results_as_a_whole(HK, H, DK, DV, L, dtype):
    """few chains, the last two cut into segments"""
    run(td.make(1 if L > 1000 else 2, L, HK, H, DK, DV, decay=0.3), dtype, reverse=L == 130)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("HK,DK", [(3, 64), (1, 128)])
def test_many_chains(HK, DK, dtype):
    """300 CTAs of 64 columns to a direction: more than two for each SM"""
    run(td.make(50, 70, HK, 3, DK, 80), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("nseq,DK,DV", [(120, 32, 16), (200, 64, 32), (290, 96, 16), (600, 32, 48)])
@pytest.mark.parametrize("dtype,reverse", [("bf16", True), ("f16", False), ("f32", False)])
def test_many_packed_sequences(nseq, DK, DV, dtype, reverse):
    """as many as a CTA has threads and more, ragged, some of no tokens"""
    rng = np.random.default_rng(nseq)
    lens = rng.integers(0, 24, nseq) * (rng.random(nseq) < 0.9)
    lens[:3] = 0, 90, 64
    cu = np.concatenate([[0], lens.cumsum()])
    run(td.make(1, int(cu[-1]), 1, 1, DK, DV), dtype, cu=cu, reverse=reverse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cu", [None, [0, 0, 40, 41, 230], [0, 2100, 2100, 2300]])
def test_scratch_of_an_earlier_call_is_not_read(cu, dtype):
    """calls on NaN before it leave NaN in the scratch that a call gets next; its bits stay the same"""
    L = cu[-1] if cu else 101
    t, _ = td.dev(td.make(1 if cu else 3, L, 1, 2, 64, 80), dtype)
    bad = {n: torch.full_like(v, float("nan")) for n, v in t.items()}
    kw = dict(cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda())
    do = torch.ones_like(t["v"])

    def call(x, d):
        o, h = binding.gated_delta_rule_fwd(**x, final_state=True, **kw)
        return [o, h, binding.gated_delta_rule_fwd(**x, **kw)[0], *binding.gated_delta_rule_bwd(**x, do=d, **kw).values()]

    want = call(t, do)
    for _ in range(2):
        assert all(v is None or torch.isnan(v).any() for v in call(bad, bad["v"]))
        got = call(t, do)
        assert all(w is None or (torch.isfinite(w).all() and torch.equal(w, v)) for w, v in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_that_grow(dtype):
    """g above 0: errors are FINE of the largest value, times what a group of 64 tokens lets grow"""
    a = td.make(2, 150, 1, 2, 64, 32)
    a["g"] = np.random.default_rng(3).uniform(-0.1, 0.2, a["g"].shape)
    t, f = td.dev(a, dtype)
    o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
    torch.cuda.synchronize()
    ro, rh, _ = onp.forward(**f, cu=[0, 150, 300])
    c = np.concatenate([np.zeros((1, 2)), f["g"].cumsum(0)])
    grow = max(float((c[i + 1:i + 65] - c[i]).max()) for i in range(300))
    td.near(o, ro, td.DT[dtype], td.FINE * np.exp(grow), td.mag(ro, f["v"]), "o")
    td.near(h, rh, torch.float32, td.FINE * np.exp(grow), td.mag(rh, f["v"]), "h_last")


@pytest.mark.gpu
def test_replaced_values_under_growth():
    """one key, beta = 1: S^T k = v whatever g; by groups errors grow with exp(64 g), token by token they do not"""
    k = torch.zeros(1, 64, 1, 32, device="cuda")
    k[..., 0] = 1
    v, one = torch.ones(1, 64, 1, 16, device="cuda"), torch.ones(1, 64, 1, device="cuda")
    o, _ = binding.gated_delta_rule_fwd(k, k, v, 0.05 * one, one, scale=1.0, final_state=True)
    torch.cuda.synchronize()
    assert float((o - 1).abs().max()) <= td.FINE * np.exp(64 * 0.05)
    state = torch.zeros(1, 1, 32, 16, device="cuda")
    for t in range(64):
        got = binding.gated_delta_rule_step(k[:, t], k[:, t], v[:, t], 2 * one[:, 0], one[:, 0], state, scale=1.0)
        # a value of 1 grows to e^2 and is taken off again: three roundings of e^2 at most
        assert float((got - 1).abs().max()) <= 3 * np.exp(2.0) * 2.0 ** -23


def c_bwd(t, do, h0, dh_last, dh0, cu=None):
    """the C call with dh0 wherever it is told, which the binding always makes itself"""
    B, L, HK, DK = t["q"].shape
    H, DV = t["v"].shape[2:]
    g = {n: torch.empty_like(t[n]) for n in ("q", "k", "v", "g", "beta")}
    p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    rc = binding.lib().gated_delta_rule_bwd(
        *(p(t[n]) for n in ("q", "k", "v", "g", "beta")), p(h0), p(do), p(dh_last),
        *(p(g[n]) for n in ("q", "k", "v", "g", "beta")), p(dh0), p(cu), B if cu is None else len(cu) - 1, L, HK, H,
        DK, DV, HK * DK, HK * DK, H * DV, DK ** -0.5, 0, binding._DTYPES[t["q"].dtype], None)
    torch.cuda.synchronize()
    assert rc == 0
    return g


# one warp to 16 columns, four warps, many chains, segments; a packed sequence of no tokens
PLACES = [("bf16", 1, 130, 1, 64, 64, None), ("f32", 1, 130, 1, 64, 48, None), ("f16", 50, 70, 3, 64, 80, None),
          ("bf16", 1, 2100, 1, 64, 64, None), ("f32", 1, 2100, 1, 32, 16, None),
          ("bf16", 1, 4500, 1, 32, 16, [0, 2200, 2200, 4500])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,B,L,H,DK,DV,cu", PLACES)
def test_states_in_place(dtype, B, L, H, DK, DV, cu):
    """h_last in h0's place and dh0 in dh_last's: the bits of separate ones"""
    t, _ = td.dev(td.make(B, L, H, H, DK, DV, decay=0.2), dtype)
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    n = B if cu is None else len(cu) - 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    h0, dh = (torch.randn(n, H, DK, DV, device="cuda", generator=gen) for _ in range(2))
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, cu_seqlens=cut, final_state=True)
    place = h0.clone()
    o1, h1 = binding.gated_delta_rule_fwd(**t, h0=place, cu_seqlens=cut, h_last=place)
    assert torch.equal(o, o1) and torch.equal(h, h1) and h1 is place
    do, apart, place = torch.ones_like(t["v"]), torch.empty_like(dh), dh.clone()
    g, g1 = c_bwd(t, do, h0, dh, apart, cut), c_bwd(t, do, h0, place, place, cut)
    assert torch.equal(apart, place) and all(torch.equal(g[m], g1[m]) for m in g)
    same = binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=dh, cu_seqlens=cut)
    assert torch.equal(apart, same["dh0"]) and torch.equal(g["q"], same["dq"])


@pytest.mark.gpu
@pytest.mark.parametrize("L", [2, 5])   # token by token, by groups
def test_more_sequences_than_a_grid_is_deep(L):
    B, last = 70000, 500
    gen = torch.Generator(device="cuda").manual_seed(L)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    t = dict(q=rn(B, L, 1, 16).bfloat16(), k=(rn(B, L, 1, 16) / 4).bfloat16(), v=rn(B, L, 1, 16).bfloat16(),
             g=-rn(B, L, 1).abs(), beta=torch.sigmoid(rn(B, L, 1)))
    do, h0 = torch.ones_like(t["v"]), rn(B, 1, 16, 16)
    end = {n: v[-last:].contiguous() for n, v in t.items()}
    o, h = binding.gated_delta_rule_fwd(**t, h0=h0, final_state=True)
    o1, h1 = binding.gated_delta_rule_fwd(**end, h0=h0[-last:].contiguous(), final_state=True)
    assert torch.equal(o[-last:], o1) and torch.equal(h[-last:], h1)
    g = binding.gated_delta_rule_bwd(**t, do=do, h0=h0, dh_last=h0)
    g1 = binding.gated_delta_rule_bwd(**end, do=do[-last:], h0=h0[-last:].contiguous(), dh_last=h0[-last:].contiguous())
    assert all(torch.equal(g[n][-last:], g1[n]) for n in g)
    if L == 2:
        one = {n: v[:, 0].contiguous() for n, v in t.items()}
        slots = torch.arange(B, dtype=torch.int32, device="cuda").flip(0).contiguous()
        slots[-1] = slots[0]   # the last row's slot has been taken by the first
        pool = h0.clone()
        o2 = binding.gated_delta_rule_step(**one, state=pool, slots=slots)
        some = h0[-last:].contiguous()
        o3 = binding.gated_delta_rule_step(**{n: v[:last].contiguous() for n, v in one.items()}, state=some,
                                           slots=(slots[:last] - (B - last)).contiguous())
        assert torch.equal(o2[:last], o3) and torch.equal(pool[-last:], some)
        assert not o2[-1].any() and torch.equal(pool[0], h0[0])


@pytest.mark.gpu
def test_calls_from_several_threads():
    """four threads with a stream each, different shapes at once: the bits of calls one by one"""
    cases = [td.dev(td.make(1, L, 1, 2, 64, 64, seed=L), d)[0] for L, d in ((300, "bf16"), (130, "f32"), (2200, "bf16"),
                                                                          (90, "f16"))]

    def call(t):
        x = t["v"].flatten(0, 1)
        o, h = binding.gated_delta_rule_fwd(**t, final_state=True)
        n, _ = binding.block_norm_fwd(o, z=t["v"], post="rms")
        gn = binding.block_norm_bwd(x, x, post="layer", w_post=torch.ones(64, device="cuda"))
        return [o, h, n, gn["dx"], gn["dw_post"], *binding.gated_delta_rule_bwd(**t, do=n).values()]

    want = [call(t) for t in cases]
    torch.cuda.synchronize()
    got = [None] * len(cases)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got[i] = call(cases[i])
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for w, g in zip(want, got):
        assert g is not None and all(a is None or torch.equal(a, b) for a, b in zip(w, g))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,L", [("bf16", 200), ("f16", 200), ("f32", 200), ("bf16", 2100), ("f32", 2100)])
@pytest.mark.parametrize("what", ["v", "k", "g", "beta"])
def test_what_is_not_finite_stays_where_it_is(dtype, L, what):
    """in one head of one sequence, from its group of 64 tokens on; its value column in v"""
    t, _ = td.dev(td.make(1, 3 * L, 2, 2, 32, 32, decay=0.2), dtype)
    cu = torch.tensor([0, L, 2 * L, 3 * L], dtype=torch.int32).cuda()
    clean, hc = binding.gated_delta_rule_fwd(**t, cu_seqlens=cu, final_state=True)
    do = torch.ones_like(clean)
    gc = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu)
    t = {n: v.clone() for n, v in t.items()}
    at = L + 150
    t[what][(0, at, 1) + ((3,) if what in "vk" else ())] = float("nan")
    o, h = binding.gated_delta_rule_fwd(**t, cu_seqlens=cu, final_state=True)
    g = binding.gated_delta_rule_bwd(**t, do=do, cu_seqlens=cu)
    torch.cuda.synchronize()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[0, L + 128:2 * L, 1, slice(3, 4) if what == "v" else slice(None)] = False
    assert torch.equal(o[keep], clean[keep]) and torch.isnan(o[0, at, 1]).any()
    assert torch.equal(h[[0, 2]], hc[[0, 2]]) and torch.equal(h[1, 0], hc[1, 0]) and torch.isnan(h[1, 1]).any()
    for n, v in g.items():
        if v is not None:
            assert torch.equal(v[:, :L], gc[n][:, :L]) and torch.equal(v[:, 2 * L:], gc[n][:, 2 * L:]), n
            assert torch.equal(v[:, :, 0], gc[n][:, :, 0]), n
            assert torch.isnan(v[0, L:at, 1]).any() or n == "dv" or what != "v", n
