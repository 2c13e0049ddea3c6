"""The FP64 references of the state-space layer's operators pinned by closed
forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import ssm_ref


def inputs(lens, H, G, N, P, seed):
    r = np.random.default_rng(seed)
    T, n = sum(lens), len(lens)
    return dict(x=r.normal(size=(T, H, P)), raw_dt=r.normal(size=(T, H)), A_log=r.normal(size=H) * 0.5,
                B=r.normal(size=(T, G, N)), C=r.normal(size=(T, G, N)), D=r.normal(size=H),
                dt_bias=r.normal(size=H) - 1, cu=np.cumsum([0] + list(lens)), state=r.normal(size=(n, H, N, P)))


def differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        at = x[i]
        x[i] = at + h
        up = f()
        x[i] = at - h
        g[i] = (up - f()) / (2 * h)
        x[i] = at
    return g


@pytest.mark.parametrize("limit", [(0.0, np.inf), (0.2, 0.6)])
def test_scan_gradients(limit):
    x = inputs([3, 0, 4], 4, 2, 3, 2, 1)
    r = np.random.default_rng(2)
    dy, dfinal = r.normal(size=x["x"].shape), r.normal(size=x["state"].shape)

    def loss():
        y, S = ssm_ref.scan(**x, limit=limit)
        return np.sum(y * dy) + np.sum(S * dfinal)

    g = ssm_ref.scan(**x, limit=limit, dy=dy, dfinal=dfinal)[2]
    for name, key in (("x", "dx"), ("raw_dt", "draw_dt"), ("A_log", "dA_log"), ("B", "dB"), ("C", "dC"),
                      ("D", "dD"), ("dt_bias", "ddt_bias"), ("state", "dinit")):
        assert np.allclose(g[key], differences(loss, x[name]), rtol=1e-6, atol=1e-7), name
    if limit[0]:
        assert np.any(g["draw_dt"] == 0) and np.any(g["draw_dt"] != 0)


def test_scan_closed_forms():
    x = inputs([6], 2, 1, 3, 4, 3)
    # no step: the state stays, y reads it
    zero = dict(x, raw_dt=np.full((6, 2), -1e4), D=None)
    y, S = ssm_ref.scan(**zero)
    assert np.array_equal(S, x["state"])
    assert np.allclose(y, np.einsum("tn,hnp->thp", x["C"][:, 0], x["state"][0]))
    # no decay: linear attention with the step sizes as weights
    lin = dict(x, A_log=np.full(2, -1e4), D=None, state=None)
    dt = ssm_ref.step_sizes(x["raw_dt"], x["dt_bias"], (0, np.inf))[0]
    w = np.tril(x["C"][:, 0] @ x["B"][:, 0].T)
    want = np.einsum("ts,sh,shp->thp", w, dt, x["x"])
    assert np.allclose(ssm_ref.scan(**lin)[0], want)
    # two sequences are two calls; a pool with slots is the same
    two = inputs([2, 4], 2, 1, 3, 4, 4)
    y, S = ssm_ref.scan(**two)
    pool = np.zeros((5, *two["state"].shape[1:]))
    pool[3], pool[1] = two["state"]
    y2, S2 = ssm_ref.scan(**dict(two, state=pool, slots=[3, 1]))
    assert np.array_equal(y, y2) and np.array_equal(S2[[3, 1]], S)
    y3, S3 = ssm_ref.scan(**dict(two, state=pool, slots=[3, -1]))
    assert np.array_equal(y3[:2], y[:2]) and np.all(y3[2:] == 0) and np.array_equal(S3[1], pool[1])


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
def test_group_norm(center, gate, act):
    if gate != "none" and act == "none":
        return
    r = np.random.default_rng(5)
    x, g, dy = r.normal(size=(3, 3, 12))
    w, b = r.normal(size=(2, 12))
    g = None if gate == "none" else g
    kw = dict(groups=3, activation=act, center=center, gate_first=gate == "first", eps=1e-3)

    def loss():
        return np.sum(ssm_ref.group_norm(x, w, b, g, **kw)["y"] * dy)

    out = ssm_ref.group_norm(x, w, b, g, **kw, dy=dy)
    for name, t in (("dx", x), ("dw", w), ("db", b), ("dgate", g)):
        if t is not None:
            assert np.allclose(out[name], differences(loss, t), rtol=1e-6, atol=1e-7), name
    if gate != "first" and center:  # groups of mean 0 and variance 1
        one = dict(kw, eps=0.0, activation="none") if g is None else None
        if one:
            y = ssm_ref.group_norm(x, np.ones(12), None, None, **one)["y"].reshape(3, 3, 4)
            assert np.allclose(y.mean(-1), 0) and np.allclose((y ** 2).mean(-1), 1)
