"""FP64 NumPy references of a state-space layer's operators (test
infrastructure only; no code shared with the GPU path): the selective scan
token by token with its hand-derived backward, also from a pool of states, and
the group norm with its activation or gate.
"""
from __future__ import annotations

import numpy as np

from . import _f64
from .layer_ref import _act, sigmoid


def step_sizes(raw_dt, dt_bias, limit):
    """(dt, d dt / d raw): the softplus clamped to `limit`, slope 0 where it holds."""
    z = _f64(raw_dt) + (0.0 if dt_bias is None else _f64(dt_bias))
    with np.errstate(invalid="ignore"):  # NaN in rows of padded sequences
        s = np.logaddexp(0.0, z)
    inside = (s > limit[0]) & (s < limit[1])
    return np.clip(s, *limit), sigmoid(z) * inside


def scan(x, raw_dt, A_log, B, C, D, dt_bias, cu, state=None, slots=None, limit=(0.0, np.inf),
         dy=None, dfinal=None):
    """y and the states left behind: S = exp(-exp(A_log) dt) S + dt B x^T,
    y = S^T C + D x, sequence n from state[slots[n]] (slots None: n; state None:
    zeros; a negative slot: zero rows). Rows of no sequence are zero. With dy
    (and dfinal) a dict of the gradients of sum(y dy) + sum(final dfinal), and
    `tall`, the step sizes' gradient with its two terms added up instead of
    taken off each other (of inputs without signs: their size)."""
    x, A, B, C = _f64(x), np.exp(_f64(A_log)), _f64(B), _f64(C)
    T, H, P = x.shape
    per, N = H // B.shape[1], B.shape[2]
    Bh, Ch = np.repeat(B, per, 1), np.repeat(C, per, 1)
    dt, slope = step_sizes(raw_dt, dt_bias, limit)
    a = np.exp(-A * dt)
    Dv = np.zeros(H) if D is None else _f64(D)
    cu = [int(c) for c in cu]
    S = np.zeros((len(cu) - 1, H, N, P)) if state is None else _f64(state).copy()
    slots = list(range(len(cu) - 1)) if slots is None else [int(s) for s in slots]
    y = np.zeros((T, H, P))
    states = {}  # of each token: the decayed state, and the one after it
    for n, sl in enumerate(slots):
        for t in range(cu[n], cu[n + 1]):
            if sl < 0:
                continue
            decayed = a[t][:, None, None] * S[sl]
            S[sl] = decayed + (dt[t][:, None] * Bh[t])[:, :, None] * x[t][:, None, :]
            if dy is not None:
                states[t] = decayed, S[sl].copy()
            y[t] = np.einsum("hn,hnp->hp", Ch[t], S[sl]) + Dv[:, None] * x[t]
    if dy is None:
        return y, S
    dy = _f64(dy)
    dS = np.zeros_like(S) if dfinal is None else _f64(dfinal).copy()
    g = {k: np.zeros_like(v) for k, v in dict(x=x, B=Bh, C=Ch, dt=dt).items()}
    dA, dD, tdt = np.zeros(H), np.zeros(H), np.zeros((T, H))
    for n in range(len(cu) - 1):
        for t in reversed(range(cu[n], cu[n + 1])):
            decayed, after = states[t]
            g["C"][t] = np.einsum("hnp,hp->hn", after, dy[t])
            dS[n] += Ch[t][:, :, None] * dy[t][:, None, :]
            Bx = np.einsum("hnp,hn,hp->h", dS[n], Bh[t], x[t])
            dl = np.sum(dS[n] * decayed, (1, 2))  # with respect to log a
            g["x"][t] = dt[t][:, None] * np.einsum("hnp,hn->hp", dS[n], Bh[t]) + Dv[:, None] * dy[t]
            g["B"][t] = dt[t][:, None] * np.einsum("hnp,hp->hn", dS[n], x[t])
            g["dt"][t] = Bx - A * dl
            tdt[t] = Bx + A * dl
            dA += -A * dt[t] * dl
            dD += np.sum(x[t] * dy[t], 1)
            dS[n] = a[t][:, None, None] * dS[n]
    draw = g["dt"] * slope
    G = B.shape[1]
    return y, S, dict(dx=g["x"], draw_dt=draw, dA_log=dA, dB=g["B"].reshape(T, G, per, N).sum(2),
                      dC=g["C"].reshape(T, G, per, N).sum(2), dD=dD, ddt_bias=draw.sum(0), dinit=dS, tall=tdt)


def group_norm(x, weight, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=True,
               gate_first=False, dy=None):
    """y, and with dy a dict of the gradients and of the sizes of what they are
    differences of (`t...`; `tz`: r (|z| + |mean|))."""
    x, w = _f64(x), _f64(weight)
    shape = x.shape
    C = shape[-1]
    x = x.reshape(-1, C)
    b = np.zeros(C) if bias is None else _f64(bias)

    def mean(v):
        return np.repeat(v.reshape(len(v), groups, -1).mean(-1), C // groups, -1)

    ga = gs = None
    if gate is not None:
        ga, gs = _act(activation, _f64(gate).reshape(-1, C))
    z = x * ga if gate_first else x
    m = mean(z) if center else np.zeros_like(z)
    r = 1 / np.sqrt(mean((z - m) ** 2) + eps)
    n = (z - m) * r
    p = n * w + b
    ya, ys = (p, 1.0) if gate_first else _act(activation, p) if gate is None else (p * ga, ga)
    tz = r * (np.abs(z) + np.abs(m))
    out = dict(y=ya.reshape(shape), tz=tz.reshape(shape))
    if dy is None:
        return out
    dy = _f64(dy).reshape(-1, C)
    dp = dy * ys
    dn = dp * w
    dz = r * (dn - n * mean(dn * n) - (mean(dn) if center else 0.0))
    out.update(dx=dz * ga if gate_first else dz, dw=np.sum(dp * n, 0), db=np.sum(dp, 0))
    if gate is not None:
        out["dgate"] = dz * x * gs if gate_first else dy * p * gs
    tdn = np.abs(dy * w) * (np.abs(ys) + (tz * np.abs(w) + np.abs(b) if gate is None and activation != "none" else 0.0))
    out["tdw"] = np.abs(dp) * tz
    rms = np.sqrt(mean(tdn ** 2))
    tdz = r * (tdn + rms * (1 + tz) * (1 + np.sqrt(mean(tz ** 2))))
    if gate_first:
        out["tdx"], out["tdgate"] = tdz * np.abs(ga), tdz * np.abs(x) * (np.abs(gs) + np.abs(ga))
    else:
        out["tdx"] = tdz
        if gate is not None:
            out["tdgate"] = np.abs(dy) * (tz * np.abs(w) + np.abs(b)) * (np.abs(gs) + np.abs(ga))
    return {k: v.reshape(shape) if v.size == x.size and v.ndim == 2 else v for k, v in out.items()}
