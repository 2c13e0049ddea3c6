"""FP64 NumPy references of the operators around the chunked one (test
infrastructure only; no code shared with the GPU path): the recurrent delta
rule from given states, the gated norm, the norms around a block and the
short causal convolution, each with hand-derived gradients where it has any.
"""
from __future__ import annotations

import numpy as np

from . import GATE_SIGMOID_BOUND, _f64


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def _gate(mode, A_log, z, lb):
    ea = np.exp(A_log)
    if mode == GATE_SIGMOID_BOUND:
        return lb * sigmoid(ea * z)
    return np.maximum(lb, -ea * np.log1p(np.exp(z)))


def recurrent(q, k, v, raw_g, A_log, dt_bias, state, cu, slots=None, raw_beta=None, raw_b=None,
              raw_w=None, scale=1.0, lower_bound=-5.0, eps=1e-6, gate_mode=GATE_SIGMOID_BOUND):
    """(o, state) with S_t = (I - kh e^T) Diag(exp g) S_{t-1} + kh w^T and
    o_t = S_t^T qh: e = beta kh, w = beta v (raw_beta), or e = b * kh,
    w = wgate * v (raw_b, raw_w). Sequence n uses state slots[n]; a negative
    slot gives zero rows. Rows of o behind the last sequence are
    NaN (not computed)."""
    q, k, v, raw_g, A_log, dt_bias = map(_f64, (q, k, v, raw_g, A_log, dt_bias))
    S = _f64(state).copy()
    T, H, K = q.shape
    o = np.full((T, H, v.shape[2]), np.nan)
    cu = [int(c) for c in cu]
    slots = list(range(len(cu) - 1)) if slots is None else [int(s) for s in slots]
    if raw_beta is not None:
        raw_beta = _f64(raw_beta)
    else:
        raw_b, raw_w = _f64(raw_b), _f64(raw_w)
    for n, sl in enumerate(slots):
        for t in range(cu[n], cu[n + 1]):
            if sl < 0:
                o[t] = 0.0
                continue
            for h in range(H):
                qh = scale * q[t, h] / np.sqrt(np.sum(q[t, h] ** 2) + eps)
                kh = k[t, h] / np.sqrt(np.sum(k[t, h] ** 2) + eps)
                g = _gate(gate_mode, A_log[h], raw_g[t, h] + dt_bias[h], lower_bound)
                if raw_beta is not None:
                    e, w = sigmoid(raw_beta[t, h]) * kh, sigmoid(raw_beta[t, h]) * v[t, h]
                else:
                    e, w = sigmoid(raw_b[t, h]) * kh, sigmoid(raw_w[t, h]) * v[t, h]
                D = np.broadcast_to(np.exp(g), (K,))[:, None] * S[sl, h]
                S[sl, h] = D - np.outer(kh, e @ D) + np.outer(kh, w)
                o[t, h] = qh @ S[sl, h]
    return o, S


def _act(kind, x):
    """(value, derivative) of the activation. 1 - s is taken as sigmoid(-x),
    which keeps its digits where s is next to 1."""
    s, c = sigmoid(x), sigmoid(-x)
    if kind == "sigmoid":
        return s, s * c
    if kind == "silu":
        return x * s, s * (1 + x * c)
    return x, np.ones_like(x)


def gated_norm(o, gate, weight, dy=None, eps=1e-6, activation="sigmoid"):
    """y = rmsnorm(o) * weight * act(gate) over the last dimension; with dy
    also (do, dgate, dweight)."""
    o, gate, weight = map(_f64, (o, gate, weight))
    r = 1 / np.sqrt(np.mean(o * o, -1, keepdims=True) + eps)
    a, da = _act(activation, gate)
    n = o * r
    y = n * weight * a
    if dy is None:
        return y
    dy = _f64(dy)
    dn = dy * weight * a
    do = r * (dn - n * np.mean(dn * n, -1, keepdims=True))
    return y, do, dy * n * weight * da, np.sum(dy * n * a, axis=tuple(range(o.ndim - 1)))


def block_norm(x, y, w_pre, w_post=None, raw_gate=None, residual_scale=1.0, eps=1e-6, dx_out=None,
               dh=None):
    """x' = x + s * sigmoid(gate) * post(y), h = rmsnorm(x') * w_pre, post(y) =
    rmsnorm(y) * w_post or y; a gate [T] or [T,D]. With dx_out and dh the
    gradients as a dict."""
    x, y, w_pre = map(_f64, (x, y, w_pre))
    a = rest = np.ones((1, 1))
    if raw_gate is not None:
        a, rest = sigmoid(_f64(raw_gate)), sigmoid(-_f64(raw_gate))  # rest = 1 - a
        a, rest = (t[:, None] if t.ndim == 1 else t for t in (a, rest))
    ry = 1 / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
    z = y * ry * _f64(w_post) if w_post is not None else y
    xo = x + residual_scale * a * z
    rx = 1 / np.sqrt(np.mean(xo * xo, -1, keepdims=True) + eps)
    n = xo * rx
    out = {"x_out": xo, "h": n * w_pre}
    if dh is None:
        return out
    dx_out, dh = _f64(dx_out), _f64(dh)
    dn = dh * w_pre
    dX = dx_out + rx * (dn - n * np.mean(dn * n, -1, keepdims=True))
    dz = residual_scale * a * dX
    out.update(dx=dX, dw_pre=np.sum(dh * n, 0))
    if w_post is None:
        out["dy"] = dz
    else:
        ny = y * ry
        dny = dz * _f64(w_post)
        out["dy"] = ry * (dny - ny * np.mean(dny * ny, -1, keepdims=True))
        out["dw_post"] = np.sum(dz * ny, 0)
    if raw_gate is not None:
        dg = residual_scale * z * dX * a * rest
        out["dgate"] = dg if _f64(raw_gate).ndim == 2 else dg.sum(1)
    return out


def short_conv(x, weight, bias, cu, init=None, activation="silu", dy=None, dfinal=None):
    """Causal depthwise convolution of each packed sequence: the rows of its
    initial state [W-1,C] (zero when None), then its tokens; y_t is the
    activation of bias + sum_j weight[:, j] * row[t + j]. Returns a dict with
    y, final (the last W-1 rows) and, with dy, the gradients."""
    x, weight = _f64(x), _f64(weight)
    C, W = weight.shape
    bias_ = np.zeros(C) if bias is None else _f64(bias)
    cu = [int(c) for c in cu]
    N = len(cu) - 1
    init = np.zeros((N, W - 1, C)) if init is None else _f64(init)
    dfinal = np.zeros((N, W - 1, C)) if dfinal is None else _f64(dfinal)
    out = {"y": np.full(x.shape, np.nan), "final": np.zeros((N, W - 1, C))}
    if dy is not None:
        dy = _f64(dy)
        out.update(dx=np.full(x.shape, np.nan), dweight=np.zeros((C, W)), dbias=np.zeros(C),
                   dinit=np.zeros((N, W - 1, C)))
    for n in range(N):
        rows = np.concatenate([init[n], x[cu[n]:cu[n + 1]]])
        m = cu[n + 1] - cu[n]
        drows = np.zeros_like(rows)
        drows[m:] += dfinal[n]
        for t in range(m):
            p = bias_ + sum(weight[:, j] * rows[t + j] for j in range(W))
            y, d = _act(activation, p)
            out["y"][cu[n] + t] = y
            if dy is not None:
                dp = dy[cu[n] + t] * d
                out["dbias"] += dp
                for j in range(W):
                    drows[t + j] += weight[:, j] * dp
                    out["dweight"][:, j] += rows[t + j] * dp
        out["final"][n] = rows[m:]
        if dy is not None:
            out["dinit"][n], out["dx"][cu[n]:cu[n + 1]] = drows[:W - 1], drows[W - 1:]
    return out
