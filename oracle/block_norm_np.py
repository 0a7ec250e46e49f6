"""NumPy float64 write-up of the block norms -- TEST INFRASTRUCTURE ONLY.

Per row:  t = (N_post(x) w_post + b_post) SiLU(z);  r' = r + s t;
y = N_pre(r') w_pre + b_pre, with N_layer(x) = (x - mean) / sqrt(var + eps),
N_rms(x) = x / sqrt(mean(x^2) + eps), and any part left out (None, or "none").
:func:`block_norm_bwd` is the plain chain rule of that definition; the norm in
front of the next block is differentiated at the r' it is given.  Pinned by
central differences of the forward in ``tests/test_block_norm.py``.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def norm(x, how, eps):
    """(normalised rows, 1 / sqrt(. + eps))"""
    if how == "layer":
        x = x - x.mean(-1, keepdims=True)
    rs = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * rs, rs


def norm_back(d, n, rs, how):
    out = d - n * (d * n).mean(-1, keepdims=True)
    if how == "layer":
        out = out - d.mean(-1, keepdims=True)
    return rs * out


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def branch(x, z, s, post, w_post, b_post, eps):
    n, rs = norm(x, post, eps) if post != "none" else (x, None)
    p = n
    if post != "none":
        p = p * (1.0 if w_post is None else w_post) + (0.0 if b_post is None else b_post)
    t = p if z is None else p * z * sigmoid(z)
    return n, rs, p, t


def block_norm_fwd(x, z=None, r=None, s=None, post="none", w_post=None, b_post=None, pre="none",
                   w_pre=None, b_pre=None, eps=1e-5):
    x, z, r, s, w_post, b_post, w_pre, b_pre = map(_f, (x, z, r, s, w_post, b_post, w_pre, b_pre))
    t = branch(x, z, s, post, w_post, b_post, eps)[3]
    r_out = (0.0 if r is None else r) + t * (1.0 if s is None else s)
    if pre == "none":
        return r_out, None
    y = norm(r_out, pre, eps)[0] * (1.0 if w_pre is None else w_pre)
    return r_out, y + (0.0 if b_pre is None else b_pre)


def block_norm_bwd(x, dr_out, dy=None, r_out=None, z=None, s=None, post="none", w_post=None,
                   b_post=None, pre="none", w_pre=None, eps=1e-5):
    """dict of dx, dz, dr, and the row sums ds, dw_post, db_post, dw_pre, db_pre; "abs" maps each
    row sum to the sum of its terms' absolute values."""
    x, dr_out, dy, r_out, z, s, w_post, b_post, w_pre = map(
        _f, (x, dr_out, dy, r_out, z, s, w_post, b_post, w_pre))
    g, terms = {}, {}
    G = np.zeros_like(x) if dr_out is None else dr_out
    if pre != "none":
        n, rs = norm(r_out, pre, eps)
        terms["dw_pre"], terms["db_pre"] = dy * n, dy
        G = G + norm_back(dy * (1.0 if w_pre is None else w_pre), n, rs, pre)
    g["dr"] = G
    n, rs, p, t = branch(x, z, s, post, w_post, b_post, eps)
    terms["ds"] = G * t
    dt = G * (1.0 if s is None else s)
    dp = dt
    if z is not None:
        sg = sigmoid(z)
        dp = dt * z * sg
        g["dz"] = dt * p * sg * (1.0 + z * (1.0 - sg))
    if post != "none":
        terms["dw_post"], terms["db_post"] = dp * n, dp
        g["dx"] = norm_back(dp * (1.0 if w_post is None else w_post), n, rs, post)
    else:
        g["dx"] = dp
    for name, v in terms.items():
        g[name] = v.reshape(-1, v.shape[-1]).sum(0)
    g["abs"] = {name: np.abs(v).reshape(-1, v.shape[-1]).sum(0) for name, v in terms.items()}
    return g
