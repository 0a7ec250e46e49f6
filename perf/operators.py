"""What is measured of the gated delta rule and of the block norms: cases,
inputs, one pass through an operator (its plain form in elementary torch
operations, or the library's call), the work a pass cannot do without, and
the operators' values from their definitions in 64 bits.

The operators (see include/ss2d.h for the full definition):

  gated delta rule, per sequence and value head, state S (DK, DV), S_0 = h0:
      d_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t)
      S_t = exp(g_t) S_{t-1} + k_t d_t^T
      o_t = scale S_t^T q_t
    kinds "fwd" (o and the last state), "bwd" (all gradients) and "step"
    (one token for each sequence, states updated in place).
  block norm, per row:
      t  = N_post(x) w_post + b_post, times SiLU(z);   r' = r + s t
      y  = N_pre(r') w_pre + b_pre
    with every part optional; kinds "norm_fwd" and "norm_bwd".
"""
import math

import torch

own = False

CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def _gdr(kind, name=None, B=1, L=1, HK=1, H=1, DK=64, DV=64, dtype="bf16", seqs=0, state=False, reverse=False,
         fused=False):
    c = dict(kind=kind, B=B, L=L, HK=HK, H=H, DK=DK, DV=DV, dtype=dtype, seqs=seqs, state=state, reverse=reverse,
             fused=fused)
    return dict(c, name=name) if name else c


def _norm(kind, name=None, rows=1, D=64, dtype="bf16", post="none", gate=False, res="none", scale=False, pre="none",
          bias=False):
    c = dict(kind=kind, rows=rows, D=D, dtype=dtype, post=post, gate=gate, res=res, scale=scale, pre=pre, bias=bias)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the mixer of a Vim-S block: 128 images of 197 tokens, inner width 768 as 12 heads of 64
        _gdr("fwd", "fwd vim-s", B=128, L=197, HK=12, H=12, DK=64, DV=64),
        # a 256 x 256 map at width 192 as one sequence: few heads, a very long chain
        _gdr("fwd", "fwd 256x256 map", B=1, L=65536, HK=3, H=3, DK=64, DV=64, state=True),
        # a packed prefill: ragged sequences continued from their states, key heads shared by value heads,
        # q, k and v views of one projection
        _gdr("fwd", "fwd packed f16", B=1, L=16384, HK=8, H=16, DK=128, DV=128, dtype="f16", seqs=24, state=True,
             fused=True),
        # the training pass of the Vim-S mixer
        _gdr("bwd", "bwd vim-s", B=128, L=197, HK=12, H=12, DK=64, DV=64),
        # the training pass at long length, wide heads, key heads shared
        _gdr("bwd", "bwd long", B=2, L=4096, HK=8, H=16, DK=128, DV=128, state=True),
        # float32 training on a few ragged sequences read from their ends, small and unequal head sizes
        _gdr("bwd", "bwd packed f32", B=1, L=1500, HK=3, H=6, DK=32, DV=64, dtype="f32", seqs=7, state=True,
             reverse=True),
        # one token of one sequence: latency
        _gdr("step", "step one", B=1, HK=12, H=12, DK=64, DV=64),
        # a full serving batch out of a pool of states
        _gdr("step", "step batch", B=256, HK=8, H=16, DK=128, DV=128),
        # the gated output norm of the Vim-S mixer, per head of 64
        _norm("norm_fwd", "norm gated heads", rows=128 * 197 * 12, D=64, post="rms", gate=True),
        # a VMamba-T stage-1 map between two blocks: layer-scaled branch added to a float32 residual, next block's
        # layer norm
        _norm("norm_fwd", "norm residual", rows=8 * 56 * 56, D=192, res="f32", scale=True, pre="layer", bias=True),
        # everything at once, forward's counterpart in training, at VMamba-B stage-3 width
        _norm("norm_bwd", "norm bwd all", rows=64 * 196, D=1024, post="rms", gate=True, res="same", scale=True,
              pre="rms"),
        # the gradient of the gated output norm on few odd rows in float32: latency
        _norm("norm_bwd", "norm bwd small", rows=197, D=191, dtype="f32", post="layer", gate=True, bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind.startswith("norm"):
        D = _log(rng, 16, 4096)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        post, pre = rng.choice([("rms", "none"), ("none", "rms"), ("none", "layer"), ("rms", "rms"),
                                ("layer", "layer"), ("layer", "none")])
        rows = _log(rng, 1, min(300000, 16_000_000 // D))
        return _norm(kind, rows=rows, D=D, dtype=dtype, post=post, gate=rng.random() < 0.5,
                     res=rng.choice(["same", "f32"]) if pre != "none" else "none",
                     scale=pre != "none" and rng.random() < 0.5, pre=pre, bias=rng.random() < 0.4)
    HK = rng.choice([1, 2, 3, 4, 6, 8, 12])
    H = HK * rng.choice([1, 1, 2, 3, 4])
    DK = rng.choice([16, 32, 48, 64, 64, 96, 128, 128])
    DV = rng.choice([16, 32, 64, 64, 80, 128, 128, 192])
    if kind == "step":
        return _gdr(kind, B=_log(rng, 1, max(1, min(512, (1 << 26) // (H * DK * DV)))), HK=HK, H=H, DK=DK, DV=DV,
                    dtype=dtype)
    tokens = _log(rng, 1, min(20000, (1 << 30) // (H * DK * DV)))
    state, reverse, fused = rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.4
    if rng.random() < 0.35:
        return _gdr(kind, B=1, L=tokens, HK=HK, H=H, DK=DK, DV=DV, dtype=dtype, seqs=rng.randint(1, 20), state=state,
                    reverse=reverse, fused=fused)
    L = _log(rng, 1, min(tokens, 8192))
    return _gdr(kind, B=max(1, tokens // L), L=L, HK=HK, H=H, DK=DK, DV=DV, dtype=dtype, state=state, reverse=reverse,
                fused=fused)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["kind"].startswith("norm"):
        R, D = c["rows"], c["D"]
        rdt = torch.float32 if c["res"] == "f32" else dt
        st["x"] = (1.5 * randn(R, D) + 0.3).to(dt)
        st["z"] = randn(R, D).to(dt) if c["gate"] else None
        st["r"] = (2.0 * randn(R, D)).to(rdt) if c["res"] != "none" else None
        st["s"] = 0.1 + 0.3 * randn(D) if c["scale"] else None
        st["w_post"] = 1.0 + 0.2 * randn(D) if c["post"] != "none" else None
        st["b_post"] = 0.2 * randn(D) if c["post"] != "none" and c["bias"] else None
        st["w_pre"] = 1.0 + 0.2 * randn(D) if c["pre"] != "none" else None
        st["b_pre"] = 0.2 * randn(D) if c["pre"] != "none" and c["bias"] else None
        if c["kind"] == "norm_bwd":
            # what a training step kept of the forward pass, and the gradients that reach the block
            t = _norm_branch(st, torch.float32)[1]
            st["r_out"] = (t if st["r"] is None else st["r"].float() + t).to(rdt)
            st["dr_out"] = randn(R, D).to(rdt)
            st["dy"] = randn(R, D).to(dt) if c["pre"] != "none" else None
        return st
    B, L, HK, H, DK, DV = (c[n] for n in ("B", "L", "HK", "H", "DK", "DV"))

    def unit(t):
        return (t / t.norm(dim=-1, keepdim=True)).to(dt)

    q, k, v = unit(randn(B, L, HK, DK)), unit(randn(B, L, HK, DK)), randn(B, L, H, DV).to(dt)
    if c["fused"]:  # views of one projection's output
        qkv = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], dim=-1)
        n = HK * DK
        q, k = qkv[..., :n].unflatten(-1, (HK, DK)), qkv[..., n:2 * n].unflatten(-1, (HK, DK))
        v = qkv[..., 2 * n:].unflatten(-1, (H, DV))
    # g = -A softplus(a + bias), softplus(bias) log-uniform in [1e-3, 1e-1], A in [1, 16]; beta = sigmoid
    dt0 = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(H, generator=gen, device="cuda"))
    A = 1 + 15 * torch.rand(H, generator=gen, device="cuda")
    g = -A * torch.nn.functional.softplus(randn(B, L, H) + torch.log(torch.expm1(dt0)))
    beta = torch.sigmoid(randn(B, L, H))
    st.update(q=q, k=k, v=v, g=g, beta=beta, cu=None, lens=None, h0=None)
    if c["kind"] == "step":
        for n in ("q", "k", "v", "g", "beta"):
            st[n] = st[n][:, 0].contiguous()
        st["pool"] = 0.5 * randn(2 * B, H, DK, DV)
        st["slots"] = torch.randperm(2 * B, generator=gen, device="cuda")[:B].to(torch.int32)
        return st
    nseq = B
    if c["seqs"]:
        nseq = c["seqs"]
        cuts = torch.randint(0, L + 1, (nseq - 1,), generator=gen, device="cuda").sort().values
        cu = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), L)])
        st["cu"], st["lens"] = cu.to(torch.int32), (cu[1:] - cu[:-1]).tolist()
    if c["state"]:
        st["h0"] = 0.5 * randn(nseq, H, DK, DV)
    if c["kind"] == "bwd":
        st["do"] = randn(B, L, H, DV).to(dt)
        st["dh"] = 0.5 * randn(nseq, H, DK, DV) if c["state"] else None
    return st


# ---------------------------------------------------------------- gated delta rule, plain
def _rows(st):
    """(index, inside): index[n, t] the token that sequence n reads at step t, with steps past its end outside."""
    c = st["case"]
    q = st["q"]
    lens = torch.tensor(st["lens"] if st["lens"] is not None else [c["L"]] * c["B"], device=q.device)
    start = lens.cumsum(0) - lens
    n = max(1, int(max(st["lens"]) if st["lens"] is not None else c["L"]))
    n = -(-n // CHUNK) * CHUNK
    t = torch.arange(n, device=q.device)
    inside = t < lens[:, None]
    idx = start[:, None] + (lens[:, None] - 1 - t if c["reverse"] else t)
    return torch.where(inside, idx, 0), inside


def _padded(x, rows, dtype=torch.float32):
    idx, inside = rows
    x = x.flatten(0, 1).to(dtype)[idx]
    return x * inside.reshape(inside.shape + (1,) * (x.dim() - 2))


def _unpadded(x, rows, like, dtype):
    idx, inside = rows
    out = torch.zeros((like.shape[0] * like.shape[1],) + tuple(x.shape[2:]), dtype=dtype, device=x.device)
    out[idx[inside]] = x[inside].to(dtype)
    return out.reshape(like.shape[:2] + x.shape[2:])


def _chunks(x):
    """(n, L, H, ...) -> (n, H, chunks, CHUNK, ...)"""
    return x.transpose(1, 2).unflatten(2, (-1, CHUNK))


def _plain_pass(st):
    """The forward pass by chunks: everything that its outputs and its gradients are made of."""
    c = st["case"]
    rows = _rows(st)
    rep = c["H"] // c["HK"]
    q, k = (_chunks(_padded(st[n], rows).repeat_interleave(rep, dim=2)) for n in ("q", "k"))
    v, g, beta = (_chunks(_padded(st[n], rows)) for n in ("v", "g", "beta"))
    beta = beta.unsqueeze(-1)
    scale = c["DK"] ** -0.5
    gam = g.cumsum(-1)
    diff = gam.unsqueeze(-1) - gam.unsqueeze(-2)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.exp(torch.where(low, diff, -math.inf))
    KK = k @ k.mT
    A = (beta * D * KK).tril(-1)
    eye = torch.eye(CHUNK, device=q.device)
    T = torch.linalg.solve_triangular(eye + A, eye.expand_as(A), upper=False, unitriangular=True)
    P = scale * D * (q @ k.mT)
    eg = torch.exp(gam).unsqueeze(-1)
    el = torch.exp(gam[..., -1:] - gam).unsqueeze(-1)
    last = eg[..., -1:, :]
    U, W = T @ (beta * v), T @ (beta * eg * k)
    kl = (el * k).mT
    n, NC = q.shape[0], q.shape[2]
    S = st["h0"].clone() if st["h0"] is not None else q.new_zeros(n, c["H"], c["DK"], c["DV"])
    Ss, Vn = [], []
    for i in range(NC):
        Ss.append(S)
        Vn.append(U[:, :, i] - W[:, :, i] @ S)
        S = last[:, :, i] * S + kl[:, :, i] @ Vn[-1]
    return dict(rows=rows, rep=rep, q=q, k=k, v=v, beta=beta, scale=scale, D=D, KK=KK, A=A, T=T, P=P, eg=eg, el=el,
                last=last, S=torch.stack(Ss, 2), Vn=torch.stack(Vn, 2), S_last=S)


def _plain_fwd(st):
    f = _plain_pass(st)
    o = f["scale"] * f["eg"] * (f["q"] @ f["S"]) + f["P"] @ f["Vn"]
    o = _unpadded(o.flatten(2, 3).transpose(1, 2), f["rows"], st["v"], st["v"].dtype)
    return [o, f["S_last"]] if st["case"]["state"] else [o]


def _plain_bwd(st):
    f = _plain_pass(st)
    q, k, v, beta, D, eg, el, last = (f[n] for n in ("q", "k", "v", "beta", "D", "eg", "el", "last"))
    S, Vn, P, T, scale = (f[n] for n in ("S", "Vn", "P", "T", "scale"))
    do = _chunks(_padded(st["do"], f["rows"]))
    NC = q.shape[2]
    PdO, qdo = P.mT @ do, (scale * eg * q).mT @ do
    bk = (beta * eg * k).mT
    dS = st["dh"] if st["dh"] is not None else torch.zeros_like(f["S_last"])
    dSs, dXs, dVns = [None] * NC, [None] * NC, [None] * NC
    for i in reversed(range(NC)):
        dSs[i] = dS
        dVn = PdO[:, :, i] + el[:, :, i] * (k[:, :, i] @ dS)
        dX = T[:, :, i].mT @ dVn
        dXs[i] = dX
        dS = last[:, :, i] * dS + qdo[:, :, i] - bk[:, :, i] @ dX
    dSs, dX = torch.stack(dSs, 2), torch.stack(dXs, 2)
    R = k @ S
    dR = -(beta * eg) * dX
    dv = beta * dX
    dP = (do @ Vn.mT).tril()
    dA = -(dX @ Vn.mT).tril(-1)
    GP = scale * D * dP
    GA = beta * D * dA
    VS = el * (Vn @ dSs.mT)
    dq = scale * eg * (do @ S.mT) + GP @ k
    dk = dR @ S.mT + VS + GP.mT @ q + (GA + GA.mT) @ k
    dbeta = (dX * (v - eg * R)).sum(-1) + (D * f["KK"] * dA).sum(-1)
    E = dP * P + dA * f["A"]
    kl = (VS * k).sum(-1)
    dgam = E.sum(-1) - E.sum(-2) + scale * (eg * (q @ S) * do).sum(-1) + (dR * R).sum(-1) - kl
    dgam[..., -1] += kl.sum(-1) + last[..., 0, 0] * (dSs * S).sum((-1, -2))
    dg = dgam.flip(-1).cumsum(-1).flip(-1)
    join = lambda x: x.flatten(2, 3).transpose(1, 2)  # noqa: E731
    group = lambda x: join(x).unflatten(2, (-1, f["rep"])).sum(3)  # noqa: E731
    out = {"dq": _unpadded(group(dq), f["rows"], st["q"], st["q"].dtype),
           "dk": _unpadded(group(dk), f["rows"], st["k"], st["k"].dtype),
           "dv": _unpadded(join(dv), f["rows"], st["v"], st["v"].dtype),
           "dg": _unpadded(join(dg), f["rows"], st["g"], torch.float32),
           "dbeta": _unpadded(join(dbeta), f["rows"], st["beta"], torch.float32)}
    if st["h0"] is not None:
        out["dh0"] = dS
    return out


def _step_values(st, dtype):
    c = st["case"]
    rep = c["H"] // c["HK"]
    q, k = (st[n].to(dtype).repeat_interleave(rep, dim=1) for n in ("q", "k"))
    slots = st["slots"].long()
    S = torch.exp(st["g"].to(dtype))[..., None, None] * st["pool"].to(dtype)[slots]
    d = st["beta"].to(dtype).unsqueeze(-1) * (st["v"].to(dtype) - (k.unsqueeze(-1) * S).sum(-2))
    S = S + k.unsqueeze(-1) * d.unsqueeze(-2)
    o = c["DK"] ** -0.5 * (q.unsqueeze(-1) * S).sum(-2)
    return o, S, slots


def _plain_step(st):
    o, S, slots = _step_values(st, torch.float32)
    st["pool"][slots] = S
    return [o.to(st["v"].dtype), st["pool"]]


# ---------------------------------------------------------------- block norms, plain
def _normed(x, how):
    """(normalised x, the factor of its rows)"""
    if how == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_branch(st, dtype):
    """s * gate * N_post(x), and the values on the way"""
    c = st["case"]
    up = lambda n: st[n].to(dtype) if st[n] is not None else None  # noqa: E731
    n, rs = _normed(up("x"), c["post"]) if c["post"] != "none" else (up("x"), None)
    p = n * up("w_post") if c["post"] != "none" else n
    if st["b_post"] is not None:
        p = p + up("b_post")
    t = p * torch.nn.functional.silu(up("z")) if c["gate"] else p
    return dict(n=n, rs=rs, p=p, t=t), t * up("s") if c["scale"] else t


def _norm_fwd_values(st, dtype):
    c = st["case"]
    t = _norm_branch(st, dtype)[1]
    r = t if st["r"] is None else st["r"].to(dtype) + t
    if c["pre"] == "none":
        return r, None
    y = _normed(r, c["pre"])[0] * st["w_pre"].to(dtype)
    return r, y + st["b_pre"].to(dtype) if st["b_pre"] is not None else y


def _plain_norm_fwd(st):
    c = st["case"]
    r, y = _norm_fwd_values(st, torch.float32)
    out = [r.to(torch.float32 if c["res"] == "f32" else st["x"].dtype)]
    return out + [y.to(st["x"].dtype)] if y is not None else out


def _norm_back(dn, n, rs, how):
    """gradient through n = normalised x"""
    d = dn - n * (dn * n).mean(-1, keepdim=True)
    return rs * (d - dn.mean(-1, keepdim=True)) if how == "layer" else rs * d


def _norm_bwd_values(st, dtype):
    c = st["case"]
    up = lambda n: st[n].to(dtype) if st[n] is not None else None  # noqa: E731
    b, _ = _norm_branch(st, dtype)
    out = {}
    dr = up("dr_out")
    if c["pre"] != "none":
        n, rs = _normed(up("r_out"), c["pre"])
        dy = up("dy")
        out["dw_pre"] = (dy * n).sum(0)
        if st["b_pre"] is not None:
            out["db_pre"] = dy.sum(0)
        dr = dr + _norm_back(dy * up("w_pre"), n, rs, c["pre"])
    if st["r"] is not None:
        out["dr"] = dr
    dt = dr
    if c["scale"]:
        out["ds"] = (dr * b["t"]).sum(0)
        dt = dr * up("s")
    dp = dt
    if c["gate"]:
        z = up("z")
        sg = torch.sigmoid(z)
        dp = dt * z * sg
        out["dz"] = dt * b["p"] * sg * (1 + z * (1 - sg))
    if c["post"] != "none":
        out["dw_post"] = (dp * b["n"]).sum(0)
        if st["b_post"] is not None:
            out["db_post"] = dp.sum(0)
        out["dx"] = _norm_back(dp * up("w_post"), b["n"], b["rs"], c["post"])
    else:
        out["dx"] = dp
    return out


def _plain_norm_bwd(st):
    out = _norm_bwd_values(st, torch.float32)
    for n, like in (("dx", "x"), ("dz", "z"), ("dr", "r")):
        if n in out:
            out[n] = out[n].to(st[like].dtype)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    st, c = state, state["case"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd}[c["kind"]](st)
    import selective_scan_ss2d_b200 as lib
    if c["kind"] == "fwd":
        o, h = lib.gated_delta_rule_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["h0"], cu_seqlens=st["cu"],
                                        reverse=c["reverse"], final_state=c["state"])
        return [o, h] if c["state"] else [o]
    if c["kind"] == "bwd":
        g = lib.gated_delta_rule_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"], st["h0"], st["dh"],
                                     cu_seqlens=st["cu"], reverse=c["reverse"])
        return {n: t for n, t in g.items() if t is not None}
    if c["kind"] == "step":
        o = lib.gated_delta_rule_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["pool"], st["slots"])
        return [o, st["pool"]]
    w = dict(z=st["z"], s=st["s"], post=c["post"], w_post=st["w_post"], b_post=st["b_post"], pre=c["pre"],
             w_pre=st["w_pre"], b_pre=st["b_pre"], eps=EPS)
    if c["kind"] == "norm_fwd":
        r_out, y = lib.block_norm_fwd(st["x"], r=st["r"], **w)
        return [r_out] if y is None else [r_out, y]
    g = lib.block_norm_bwd(st["x"], st["dr_out"], st["dy"], r_out=st["r_out"], residual=c["res"] != "none", **w)
    return {n: t for n, t in g.items() if t is not None}


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["kind"].startswith("norm"):
        n = c["rows"] * c["D"]
        re = 4 if c["res"] == "f32" else e
        has_r, has_y, gate = c["res"] != "none", c["pre"] != "none", c["gate"]
        if c["kind"] == "norm_fwd":  # x, z, r read; r' and y written
            return {"bytes": n * (e + e * gate + re * has_r + re + e * has_y), "flops": 12.0 * n}
        # x, z, dr', dy and (for the second norm) r' read; dx, dz, dr written
        return {"bytes": n * (2 * e + 2 * e * gate + re + re * has_r + (e + re) * has_y), "flops": 30.0 * n}
    tok = c["B"] * c["L"]
    n = c["B"] * (1 if c["kind"] == "step" or not c["seqs"] else c["seqs"])
    S = 4 * n * c["H"] * c["DK"] * c["DV"]
    qk, v, gb = 2 * tok * c["HK"] * c["DK"] * e, tok * c["H"] * c["DV"] * e, 8 * tok * c["H"]
    upd = tok * c["H"] * c["DK"] * c["DV"]
    if c["kind"] == "step":
        return {"bytes": qk + 2 * v + gb + 2 * S, "flops": 7.0 * upd}
    if c["kind"] == "fwd":  # k.S, the rank-one update, q.S
        return {"bytes": qk + 2 * v + gb + 2 * S * c["state"], "flops": 6.0 * upd}
    # the states once more (4), then do.S, S.p, dS.k, dS.d and the two rank-one updates of dS (12)
    return {"bytes": 2 * qk + 3 * v + 2 * gb + 3 * S * c["state"], "flops": 16.0 * upd}


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_steps(st):
    """The recurrence token by token: yields per step what the definition names."""
    c = st["case"]
    rows = _rows(st)
    rep = c["H"] // c["HK"]
    w = torch.float64
    q, k = (_padded(st[n], rows, w).repeat_interleave(rep, dim=2) for n in ("q", "k"))
    v, g, beta = (_padded(st[n], rows, w) for n in ("v", "g", "beta"))
    S = (st["h0"].to(w) if st["h0"] is not None else
         torch.zeros(q.shape[0], c["H"], c["DK"], c["DV"], dtype=w, device=q.device))
    return rows, q, k, v, torch.exp(g), beta, S


def _exact_next(S, a, k, v, beta):
    aS = a[..., None, None] * S
    kS = torch.einsum("bhk,bhkv->bhv", k, aS)
    d = beta.unsqueeze(-1) * (v - kS)
    return aS + k.unsqueeze(-1) * d.unsqueeze(-2), aS, kS, d


def _longest(st):
    return max(st["lens"]) if st["lens"] is not None else st["case"]["L"]


def _exact_fwd(st):
    rows, q, k, v, a, beta, S = _exact_steps(st)
    o = torch.zeros_like(v)
    for t in range(_longest(st)):
        S = _exact_next(S, a[:, t], k[:, t], v[:, t], beta[:, t])[0]
        o[:, t] = torch.einsum("bhk,bhkv->bhv", q[:, t], S)
    o = _unpadded(o * st["case"]["DK"] ** -0.5, rows, st["v"], torch.float64)
    return [o, S] if st["case"]["state"] else [o]


def _exact_bwd(st):
    c = st["case"]
    rows, q, k, v, a, beta, S = _exact_steps(st)
    do = _padded(st["do"], rows, torch.float64)
    n, sc, part = _longest(st), c["DK"] ** -0.5, 64
    keep = {}
    for t in range(n):
        if t % part == 0:
            keep[t] = S
        S = _exact_next(S, a[:, t], k[:, t], v[:, t], beta[:, t])[0]
    dS = st["dh"].to(torch.float64) if st["dh"] is not None else torch.zeros_like(S)
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, a, beta))
    for t0 in sorted(keep, reverse=True):
        S, mid = keep.pop(t0), []
        for t in range(t0, min(t0 + part, n)):
            mid.append((S,) + _exact_next(S, a[:, t], k[:, t], v[:, t], beta[:, t]))
            S = mid[-1][1]
        for t in reversed(range(t0, min(t0 + part, n))):
            S0, S1, aS, kS, d = mid.pop()
            dS = dS + sc * q[:, t].unsqueeze(-1) * do[:, t].unsqueeze(-2)
            dq[:, t] = sc * torch.einsum("bhkv,bhv->bhk", S1, do[:, t])
            dd = torch.einsum("bhkv,bhk->bhv", dS, k[:, t])
            p = beta[:, t].unsqueeze(-1) * dd
            dk[:, t] = torch.einsum("bhkv,bhv->bhk", dS, d) - torch.einsum("bhkv,bhv->bhk", aS, p)
            dv[:, t] = p
            db[:, t] = (dd * (v[:, t] - kS)).sum(-1)
            daS = dS - k[:, t].unsqueeze(-1) * p.unsqueeze(-2)
            dg[:, t] = (daS * aS).sum((-1, -2))
            dS = a[:, t][..., None, None] * daS
    group = lambda x: x.unflatten(2, (c["HK"], -1)).sum(3)  # noqa: E731
    w = torch.float64
    out = {"dq": _unpadded(group(dq), rows, st["q"], w), "dk": _unpadded(group(dk), rows, st["k"], w),
           "dv": _unpadded(dv, rows, st["v"], w), "dg": _unpadded(dg, rows, st["g"], w),
           "dbeta": _unpadded(db, rows, st["beta"], w)}
    if st["h0"] is not None:
        out["dh0"] = dS
    return out


def _exact_step(st):
    w = torch.float64
    rep = st["case"]["H"] // st["case"]["HK"]
    slots = st["slots"].long()
    q, k = (st[n].to(w).repeat_interleave(rep, dim=1) for n in ("q", "k"))
    pool = st["pool"].to(w)
    S = _exact_next(pool[slots], torch.exp(st["g"].to(w)), k, st["v"].to(w), st["beta"].to(w))[0]
    pool[slots] = S
    return [st["case"]["DK"] ** -0.5 * torch.einsum("bhk,bhkv->bhv", q, S), pool]


def _exact_norm(x, how, w, b):
    n = x - x.mean(-1, keepdim=True) if how == "layer" else x
    n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + EPS) * w
    return n + b if b is not None else n


def _exact_block(st, leaves):
    c, g = st["case"], lambda n: leaves.get(n)  # noqa: E731
    t = _exact_norm(g("x"), c["post"], g("w_post"), g("b_post")) if c["post"] != "none" else g("x")
    if c["gate"]:
        t = t * g("z") / (1 + torch.exp(-g("z")))
    if c["scale"]:
        t = t * g("s")
    return t


def _exact_norm_case(st):
    c, w = st["case"], torch.float64
    names = ("x", "z", "s", "w_post", "b_post", "w_pre", "b_pre")
    leaf = {n: st[n].to(w) for n in names if st[n] is not None}
    if c["kind"] == "norm_fwd":
        t = _exact_block(st, leaf)
        r = t if st["r"] is None else st["r"].to(w) + t
        return [r] if c["pre"] == "none" else [r, _exact_norm(r, c["pre"], leaf["w_pre"], leaf.get("b_pre"))]
    # the gradients by differentiation: the second norm at the residual that the forward kept, then the branch
    for n in leaf:
        leaf[n].requires_grad_(True)
    out, dr = {}, st["dr_out"].to(w)
    if c["pre"] != "none":
        r = st["r_out"].to(w).requires_grad_(True)
        _exact_norm(r, c["pre"], leaf["w_pre"], leaf.get("b_pre")).backward(st["dy"].to(w))
        dr = dr + r.grad
    _exact_block(st, leaf).backward(dr)
    if st["r"] is not None:
        out["dr"] = dr
    return dict(out, **{"d" + n: t.grad for n, t in leaf.items()})


def exact(case, seed):
    if case["kind"] != "step" and not case["kind"].startswith("norm") and case["L"] > 100000:
        return None
    st = prepare(case, seed)
    return {"fwd": _exact_fwd, "bwd": _exact_bwd, "step": _exact_step}.get(case["kind"], _exact_norm_case)(st)
