"""Pins of the FP64 references of the operators around the chunked one
(oracle/layer_ref.py): the recurrent form against the token recurrences of
the KDA and GDN-2 oracles, and every gradient against central differences.
"""
import numpy as np
import pytest

import oracle
from oracle import layer_ref

RNG = np.random.default_rng


def draw(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("mode", [0, 1])
def test_recurrent_is_the_kda_oracle_from_a_state(per_head, mode):
    rng = RNG(1)
    T, H, K, cu = 9, 2, 8, [0, 4, 4, 9]
    g = (T, H) if per_head else (T, H, K)
    q, k, v, raw_g, rb = draw(rng, T, H, K), draw(rng, T, H, K), draw(rng, T, H, K), draw(rng, *g), draw(rng, T, H)
    A, dt, h0 = draw(rng, H), draw(rng, *g[1:]), draw(rng, 3, H, K, K)
    o, S = layer_ref.recurrent(q, k, v, raw_g, A, dt, h0, cu, raw_beta=rb, gate_mode=mode, scale=0.7)
    ref = oracle.kda(q, k, v, raw_g, rb, A, dt, cu_seqlens=cu, h0=h0, gate_mode=mode, scale=0.7)
    np.testing.assert_allclose(o, ref["o"], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(S, ref["ht"], rtol=1e-12, atol=1e-13)


def test_recurrent_gdn2_is_its_oracle_and_reduces_to_kda():
    rng = RNG(2)
    T, H, K, cu = 7, 2, 8, [0, 3, 7]
    q, k, v, g, b, w = (draw(rng, T, H, K) for _ in range(6))
    A, dt = draw(rng, H), draw(rng, H, K)
    o, _ = layer_ref.recurrent(q, k, v, g, A, dt, np.zeros((2, H, K, K)), cu, raw_b=b, raw_w=w)
    np.testing.assert_allclose(o, oracle.gdn2(q, k, v, g, b, w, A, dt, cu_seqlens=cu)["o"],
                               rtol=1e-12, atol=1e-13)
    beta, h0 = draw(rng, T, H), draw(rng, 2, H, K, K)
    wide = np.repeat(beta[:, :, None], K, 2)
    a = layer_ref.recurrent(q, k, v, g, A, dt, h0, cu, raw_b=wide, raw_w=wide)
    b = layer_ref.recurrent(q, k, v, g, A, dt, h0, cu, raw_beta=beta)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-13)


def test_recurrent_slots_and_padding():
    rng = RNG(3)
    T, H, K = 5, 1, 8
    q, k, v, g = (draw(rng, T, H, K) for _ in range(4))
    beta, A, dt, pool = draw(rng, T, H), draw(rng, H), draw(rng, H, K), draw(rng, 4, H, K, K)
    o, S = layer_ref.recurrent(q, k, v, g, A, dt, pool, [0, 2, 3, 3, 4], [3, -1, 2, 0], raw_beta=beta)
    assert np.all(o[2] == 0) and np.isnan(o[4]).all()
    assert np.array_equal(S[1:3], pool[1:3])
    for sl, a, b in ((3, 0, 2), (0, 3, 4)):
        ref = oracle.kda(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], A, dt, h0=pool[sl:sl + 1])
        np.testing.assert_allclose(S[sl], ref["ht"][0], rtol=1e-12, atol=1e-13)


def differences(f, x, eps=1e-6):
    """Central differences of the scalar f with respect to every element."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        up = f()
        x[i] = old - eps
        dn = f()
        x[i] = old
        g[i] = (up - dn) / (2 * eps)
    return g


def agree(got, want):
    np.testing.assert_allclose(got, want, rtol=2e-7, atol=2e-8)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_norm_gradients(act):
    rng = RNG(4)
    o, g, w, dy = draw(rng, 3, 2, 8), draw(rng, 3, 2, 8), draw(rng, 8), draw(rng, 3, 2, 8)
    grads = layer_ref.gated_norm(o, g, w, dy, activation=act)[1:]
    loss = lambda: np.sum(layer_ref.gated_norm(o, g, w, activation=act) * dy)  # noqa: E731
    for got, x in zip(grads, (o, g, w)):
        agree(got, differences(loss, x))


@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradients(gate, post):
    rng = RNG(5)
    x, y, w, dxo, dh = draw(rng, 3, 8), draw(rng, 3, 8), draw(rng, 8), draw(rng, 3, 8), draw(rng, 3, 8)
    wp = draw(rng, 8) if post else None
    g = {None: None, "token": draw(rng, 3), "channel": draw(rng, 3, 8)}[gate]
    run = lambda **kw: layer_ref.block_norm(x, y, w, wp, g, 0.3, **kw)  # noqa: E731
    r = run(dx_out=dxo, dh=dh)

    def loss():
        a = run()
        return np.sum(a["x_out"] * dxo) + np.sum(a["h"] * dh)

    for name, leaf in (("dx", x), ("dy", y), ("dw_pre", w), ("dw_post", wp), ("dgate", g)):
        if leaf is not None:
            agree(r[name], differences(loss, leaf))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_short_conv_gradients(W, act):
    rng = RNG(6)
    cu, C = [0, 1, 1, 6, 8], 3
    x, w, b, init = draw(rng, 8, C), draw(rng, C, W), draw(rng, C), draw(rng, 4, W - 1, C)
    dy, df = draw(rng, 8, C), draw(rng, 4, W - 1, C)
    r = layer_ref.short_conv(x, w, b, cu, init, act, dy, df)

    def loss():
        a = layer_ref.short_conv(x, w, b, cu, init, act)
        return np.sum(a["y"] * dy) + np.sum(a["final"] * df)

    for name, leaf in (("dx", x), ("dweight", w), ("dbias", b), ("dinit", init)):
        agree(r[name], differences(loss, leaf))


def test_short_conv_in_two_parts_is_one():
    rng = RNG(7)
    x, w, b = draw(rng, 9, 4), draw(rng, 4, 4), draw(rng, 4)
    whole = layer_ref.short_conv(x, w, b, [0, 9])
    first = layer_ref.short_conv(x[:5], w, b, [0, 5])
    second = layer_ref.short_conv(x[5:], w, b, [0, 4], first["final"])
    np.testing.assert_allclose(np.concatenate([first["y"], second["y"]]), whole["y"], rtol=1e-13)
    assert np.array_equal(second["final"], whole["final"])


def test_gate_slopes_keep_their_digits_far_from_zero():
    x = np.array([-700.0, -40.0, -17.0, 17.0, 40.0, 700.0])
    want = np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))) ** 2
    np.testing.assert_allclose(layer_ref._act("sigmoid", x)[1], want, rtol=1e-14)
    one, zero = np.ones((6, 1)), np.zeros((6, 1))
    got = layer_ref.block_norm(zero, one, np.ones(1), None, x, 1.0, dx_out=one, dh=zero)["dgate"]
    np.testing.assert_allclose(got, want, rtol=1e-14)
