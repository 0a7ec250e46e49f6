"""NumPy float64 write-up of the gated delta rule -- TEST INFRASTRUCTURE ONLY.

Token by token, per sequence and value head (key head h // (H // HK)), S_0 = h0 or 0:

    d_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t)
    S_t = exp(g_t) S_{t-1} + k_t d_t^T
    o_t = scale S_t^T q_t

:func:`forward` and :func:`backward` take the packed layout (tokens, heads, size) and
the sequences' first tokens; :func:`backward` is the reverse sweep of those
three lines with every state kept.  Pinned in ``tests/test_gated_delta.py`` by
central differences, by the identity S^T k = v of an undecayed full
update, and against the selective reading of an orthonormal key set.
"""
from __future__ import annotations

import numpy as np


def order(cu, n, reverse):
    """tokens of sequence n in the order they are read"""
    r = np.arange(cu[n], cu[n + 1])
    return r[::-1] if reverse else r


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def forward(q, k, v, g, beta, cu, h0=None, scale=None, reverse=False):
    """q, k (T, HK, DK), v (T, H, DV), g, beta (T, H), cu (nseq + 1) -> o (T, H, DV), h_last, states: list per
    sequence of S before each token and after the last"""
    q, k, v, g, beta, h0 = map(_f, (q, k, v, g, beta, h0))
    T, HK, DK = q.shape
    H, DV = v.shape[1:]
    rep = H // HK
    scale = DK ** -0.5 if scale is None else scale
    nseq = len(cu) - 1
    o = np.zeros((T, H, DV))
    h = np.zeros((nseq, H, DK, DV))
    states = []
    for n in range(nseq):
        S = h0[n].copy() if h0 is not None else np.zeros((H, DK, DV))
        kept = [S]
        for t in order(cu, n, reverse):
            kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
            a = np.exp(g[t])[:, None, None]
            d = beta[t][:, None] * (v[t] - (a * S * kt[:, :, None]).sum(1))
            S = a * S + kt[:, :, None] * d[:, None, :]
            o[t] = scale * (S * qt[:, :, None]).sum(1)
            kept.append(S)
        h[n] = S
        states.append(kept)
    return o, h, states


def backward(q, k, v, g, beta, cu, do, h0=None, dh_last=None, scale=None, reverse=False):
    q, k, v, g, beta, h0, do, dh_last = map(_f, (q, k, v, g, beta, h0, do, dh_last))
    T, HK, DK = q.shape
    H, DV = v.shape[1:]
    rep = H // HK
    scale = DK ** -0.5 if scale is None else scale
    _, _, states = forward(q, k, v, g, beta, cu, h0, scale, reverse)
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g),
           "dbeta": np.zeros_like(g), "dh0": np.zeros((len(cu) - 1, H, DK, DV))}
    for n in range(len(cu) - 1):
        dS = dh_last[n].copy() if dh_last is not None else np.zeros((H, DK, DV))
        seq = order(cu, n, reverse)
        for i in reversed(range(len(seq))):
            t = seq[i]
            S0, S1 = states[n][i], states[n][i + 1]
            kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
            a = np.exp(g[t])[:, None, None]
            dS = dS + scale * qt[:, :, None] * do[t][:, None, :]
            dq = scale * (S1 * do[t][:, None, :]).sum(2)
            u = v[t] - (a * S0 * kt[:, :, None]).sum(1)     # d = beta u
            dd = (dS * kt[:, :, None]).sum(1)
            p = beta[t][:, None] * dd                       # gradient of u
            dk = (dS * (beta[t][:, None] * u)[:, None, :]).sum(2) - (a * S0 * p[:, None, :]).sum(2)
            out["dq"][t] = dq.reshape(HK, rep, DK).sum(1)
            out["dk"][t] = dk.reshape(HK, rep, DK).sum(1)
            out["dv"][t] = p
            out["dbeta"][t] = (dd * u).sum(1)
            daS = dS - kt[:, :, None] * p[:, None, :]
            out["dg"][t] = (daS * a * S0).sum((1, 2))
            dS = a * daS
        out["dh0"][n] = dS
    return out
