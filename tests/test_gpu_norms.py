"""GPU parity of the gated norm and the block norm, forward and backward,
against the FP64 reference (needs an MI355X).

Tolerances. Every output is fp32 arithmetic rounded once: half a step of the
dtype per element (2^-8 of the value for bf16) plus the fp32 error of the
terms it is formed from. A row's sums run over at most 8192 terms in a tree
of serial runs of 16 and 13 levels, so they carry at most 29 roundings of
2^-24, the factors (rsqrt, sigmoid, products) about 12 more: 41 * 2^-24 =
2.5e-6 of the terms' size, for which 4e-6 of the element's own term plus
4e-6 of the row's root mean square is allowed (of a difference such as
dn - n mean(dn n) the first part has the size of dn, the second that of the
row). Parameter gradients are sums over rows, each term with the error above,
in fp32: normalised L2 1e-5.
"""
import numpy as np
import pytest
import torch

from oracle import layer_ref
from recompute_kda_chunked_amd import (block_norm, block_norm_backward, block_norm_forward,
                                       gated_norm, gated_norm_backward, gated_norm_forward)
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def check(name, got, ref, dtype, terms=None):
    """Elements of `got` within the rounding of the dtype and 4e-6 of their
    value and of their row's root mean square (or those of the `terms` they
    are the difference of)."""
    got, ref = to_np(got), np.asarray(ref)
    terms = np.abs(ref if terms is None else np.asarray(terms))
    scale = terms + np.sqrt(np.mean(terms ** 2, -1, keepdims=True))
    off = np.abs(got - ref) - HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-5) - 4e-6 * scale
    print("%s worst excess %.2e L2 %.2e" % (name, off.max() if off.size else 0, rel(got, ref)), flush=True)
    assert np.isfinite(got).all() and np.all(off <= 0), name


def randn(seed, dtype, *shape, scale=1.0, shift=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dtype)


# ------------------------------------------------------------------ gated norm


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [64, 128, 256])
@pytest.mark.parametrize("rows", [(1, 1), (3, 5), (67, 2), (700, 8)])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_norm(dtype, V, rows, act):
    announce("gated norm %s V%d rows %s %s" % (dtype, V, rows, act))
    o, g, dy = (randn(s, dtype, *rows, V, scale=2.0) for s in (1, 2, 3))
    w = randn(4, F32, V, scale=0.3, shift=1.0)
    y, do, dg, dw = layer_ref.gated_norm(o, g, w, dy, activation=act)
    check("y", gated_norm_forward(o, g, w, activation=act), y, dtype)
    got = gated_norm_backward(o, g, w, dy, activation=act)
    r = 1 / np.sqrt(np.mean(to_np(o) ** 2, -1, keepdims=True) + 1e-6)
    a = layer_ref._act(act, to_np(g))[0]
    check("do", got[0], do, dtype, terms=r * to_np(dy) * to_np(w) * a)
    check("dgate", got[1], dg, dtype)
    assert got[2].dtype is F32 and rel(to_np(got[2]), dw) <= 1e-5


def test_gated_norm_small_and_zero_rows():
    announce("gated norm, rows of zeros and of tiny values")
    o = randn(5, F32, 6, 2, 64)
    o[0], o[1] = 0.0, o[1] * 1e-20
    o[2] *= 1e15
    g, dy, w = randn(6, F32, 6, 2, 64, scale=30.0), randn(7, F32, 6, 2, 64), randn(8, F32, 64)
    y, do, dg, dw = layer_ref.gated_norm(o, g, w, dy)
    got = (gated_norm_forward(o, g, w), *gated_norm_backward(o, g, w, dy))
    for name, a, b in zip(("y", "do", "dgate", "dweight"), got, (y, do, dg, dw)):
        assert np.isfinite(to_np(a)).all() and rel(to_np(a), b) <= 1e-5, name
    assert bool((got[0][0] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_norm_autograd_and_repeat(dtype):
    announce("gated norm autograd %s" % dtype)
    leaves = [randn(9, dtype, 33, 4, 128), randn(10, dtype, 33, 4, 128), randn(11, F32, 128)]
    for t in leaves:
        t.requires_grad_(True)
    y = gated_norm(*leaves, activation="silu")
    dy = randn(12, dtype, 128, 33, 4).permute(1, 2, 0)  # not contiguous
    y.backward(dy)
    want = gated_norm_backward(*[t.detach() for t in leaves], dy.contiguous(), activation="silu")
    again = gated_norm_backward(*[t.detach() for t in leaves], dy.contiguous(), activation="silu")
    for t, a, b in zip(leaves, want, again):
        assert torch.equal(t.grad, a) and torch.equal(a, b)
    with torch.no_grad():
        assert torch.equal(gated_norm(*leaves, activation="silu"), y)


# ------------------------------------------------------------------ block norm


def block_inputs(dtype, T, D, gate, post, seed):
    x, y, dxo, dh = (randn(seed + s, dtype, T, D, scale=1.5) for s in range(4))
    wp = randn(seed + 4, F32, D, scale=0.3, shift=1.0)
    wq = randn(seed + 5, F32, D, scale=0.3, shift=1.0) if post else None
    g = {"none": None, "token": randn(seed + 6, dtype, T), "channel": randn(seed + 6, dtype, T, D)}[gate]
    return x, y, wp, wq, g, dxo, dh


def block_check(dtype, x, y, wp, wq, g, dxo, dh, s=0.3):
    kw = dict(w_post=wq, raw_gate=g, residual_scale=s)
    ref = layer_ref.block_norm(x, y, wp, wq, g, s, dx_out=np.zeros(x.shape) if dxo is None else dxo,
                               dh=np.zeros(x.shape) if dh is None else dh)
    xo, h = block_norm_forward(x, y, wp, **kw)
    check("x_out", xo, ref["x_out"], dtype)
    check("h", h, ref["h"], dtype)
    dx, dy, dwp, dwq, dg = block_norm_backward(x, y, wp, dxo, dh, **kw)
    # dx is dx_out plus a difference whose terms are of the size of rx dh w
    rx = 1 / np.sqrt(np.mean(ref["x_out"] ** 2, -1, keepdims=True) + 1e-6)
    zero = np.zeros(x.shape)
    dxt = np.abs(zero if dxo is None else to_np(dxo)) + rx * np.abs((zero if dh is None else to_np(dh)) * to_np(wp))
    check("dx", dx, ref["dx"], dtype, terms=dxt)
    a = np.ones((1, 1)) if g is None else layer_ref.sigmoid(to_np(g))
    a = a[:, None] if a.ndim == 1 else a
    ry = 1 / np.sqrt(np.mean(to_np(y) ** 2, -1, keepdims=True) + 1e-6)
    check("dy", dy, ref["dy"], dtype, terms=dxt * a * s * (1.0 if wq is None else ry * np.abs(to_np(wq))))
    z = to_np(y) if wq is None else to_np(y) * ry * to_np(wq)
    if g is not None and g.dim() == 2:
        check("dgate", dg, ref["dgate"], dtype, terms=s * z * dxt * a * (1 - a))
    elif g is not None:  # one sum over the row: its terms add up in magnitude
        off = np.abs(to_np(dg) - ref["dgate"]) - HALF_STEP[dtype] * np.abs(ref["dgate"]) * (1 + 1e-5)
        assert np.all(off <= 4e-6 * np.sum(np.abs(s * z * dxt * a * (1 - a)), -1))
    else:
        assert dg is None
    assert rel(to_np(dwp), ref["dw_pre"]) <= 1e-5
    assert dwq is None if wq is None else rel(to_np(dwq), ref["dw_post"]) <= 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D", [(1, 8), (5, 264), (3, 2048), (130, 2056), (2, 8192), (900, 512)])
def test_block_norm(dtype, gate, post, T, D):
    announce("block norm %s gate %s post %s T%d D%d" % (dtype, gate, post, T, D))
    block_check(dtype, *block_inputs(dtype, T, D, gate, post, 20))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_norm_with_one_output_gradient(dtype):
    announce("block norm, one output unused %s" % dtype)
    for which in (5, 6):
        v = list(block_inputs(dtype, 7, 328, "channel", True, 30))
        v[which] = None
        block_check(dtype, *v)
    x, y, wp, wq, g, dxo, dh = block_inputs(dtype, 7, 328, "channel", True, 30)
    got = block_norm_backward(x, y, wp, None, dh, w_post=wq, raw_gate=g)
    want = block_norm_backward(x, y, wp, torch.zeros_like(x), dh, w_post=wq, raw_gate=g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_block_norm_autograd_and_repeat(dtype, gate):
    announce("block norm autograd %s %s" % (dtype, gate))
    x, y, wp, wq, g, dxo, dh = block_inputs(dtype, 1100, 264, gate, True, 40)
    leaves = [t for t in (x, y, wp, wq, g) if t is not None]
    kw = dict(w_post=wq, raw_gate=g, residual_scale=0.7)
    want = block_norm_backward(x, y, wp, dxo, dh, **kw)
    again = block_norm_backward(x, y, wp, dxo, dh, **kw)
    for t in leaves:
        t.requires_grad_(True)
    xo, h = block_norm(x, y, wp, **kw)
    torch.autograd.backward((xo, h), (dxo, dh))
    for t, a, b in zip(leaves, [w for w in want if w is not None], [w for w in again if w is not None]):
        assert torch.equal(t.grad, a) and torch.equal(a, b)
    for t in leaves:
        t.grad = None
    block_norm(x, y, wp, **kw)[1].backward(dh)  # x_out unused
    assert torch.equal(x.grad, block_norm_backward(x, y, wp, None, dh, **kw)[0])


def test_no_rows():
    announce("norms of no rows")
    w = randn(50, F32, 64)
    o = torch.empty((0, 3, 64), device="cuda")
    assert gated_norm_forward(o, o, w).shape == o.shape
    do, dg, dw = gated_norm_backward(o, o, w, o)
    assert do.shape == o.shape and bool((dw == 0).all())
    x = torch.empty((0, 64), device="cuda")
    assert block_norm_forward(x, x, w)[1].shape == (0, 64)
    got = block_norm_backward(x, x, w, x, x, w_post=w, raw_gate=x)
    assert bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_norms_captured_and_replayed():
    announce("norms in a graph")
    o, g, dy, w = (randn(60, BF16, 300, 2, 128), randn(61, BF16, 300, 2, 128), randn(62, BF16, 300, 2, 128),
                   randn(63, F32, 128))
    x, y, wp, wq, gt, dxo, dh = block_inputs(BF16, 300, 1024, "channel", True, 64)

    def step():
        return (gated_norm_forward(o, g, w), *gated_norm_backward(o, g, w, dy),
                *block_norm_forward(x, y, wp, w_post=wq, raw_gate=gt),
                *block_norm_backward(x, y, wp, dxo, dh, w_post=wq, raw_gate=gt))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        o.mul_(1.25)
        x.mul_(0.75)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_norms_on_another_stream():
    announce("norms on a stream of their own")
    o, g, w, dy = randn(70, F32, 65, 3, 64), randn(71, F32, 65, 3, 64), randn(72, F32, 64), randn(73, F32, 65, 3, 64)
    want = (gated_norm_forward(o, g, w), *gated_norm_backward(o, g, w, dy))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = (gated_norm_forward(o, g, w), *gated_norm_backward(o, g, w, dy))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_larger_than_the_caches(dtype):
    announce("norms past the caches %s" % dtype)  # 400 MB and more per launch
    T = 8192 if dtype is BF16 else 4096
    o, g, dy, w = randn(80, dtype, T, 64, 128), randn(81, dtype, T, 64, 128), randn(82, dtype, T, 64, 128), randn(83, F32, 128)
    y, got = gated_norm_forward(o, g, w), gated_norm_backward(o, g, w, dy)
    dw = torch.zeros(128, dtype=torch.float64, device="cuda")
    for a in range(0, T, 700):  # the same rows in smaller launches
        s = slice(a, min(a + 700, T))
        assert torch.equal(y[s], gated_norm_forward(o[s], g[s], w))
        part = gated_norm_backward(o[s], g[s], w, dy[s])
        assert torch.equal(got[0][s], part[0]) and torch.equal(got[1][s], part[1])
        dw += part[2].double()
    assert rel(to_np(got[2]), to_np(dw)) <= 1e-5
    del o, g, dy, y, got, part
    for gate, post in (("channel", True), ("token", False), ("none", True)):
        x, y, wp, wq, gt, dxo, dh = block_inputs(dtype, 2 * T, 4096, gate, post, 84)
        kw = dict(w_post=wq, residual_scale=0.4)
        out, got = block_norm_forward(x, y, wp, raw_gate=gt, **kw), block_norm_backward(x, y, wp, dxo, dh, raw_gate=gt, **kw)
        dwp = torch.zeros(4096, dtype=torch.float64, device="cuda")
        for a in range(0, 2 * T, 900):
            s = slice(a, min(a + 900, 2 * T))
            gs = None if gt is None else gt[s].clone()
            assert all(torch.equal(u[s], v) for u, v in zip(out, block_norm_forward(x[s], y[s], wp, raw_gate=gs, **kw)))
            part = block_norm_backward(x[s], y[s], wp, dxo[s], dh[s], raw_gate=gs, **kw)
            assert torch.equal(got[0][s], part[0]) and torch.equal(got[1][s], part[1])
            assert gt is None or torch.equal(got[4][s], part[4])
            dwp += part[2].double()
        assert rel(to_np(got[2]), to_np(dwp)) <= 1e-5


# ------------------------------------------------------------------ gates far from zero


def far_gates(seed, dtype, lo, hi, *shape):
    """Gates of lo .. hi in magnitude, of both signs."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = lo + (hi - lo) * torch.rand(shape, generator=gen, device="cuda")
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.5, -g, g).to(dtype)


# The slope s(g) (1 - s(g)) of a gate of magnitude m is e^-m to within e^-m, so
# its relative error is that of an exponential: half a step of m log2(e) (up to
# 16: 2^-20, up to 40: 2^-19) times ln 2, and m times the constant's 1.3e-8,
# 0.9e-6 and 1.8e-6 in all. With the 2.5e-6 of the other factors (see above):
# 3.4e-6 and 4.3e-6 of the element's value.
FAR = [(8.0, 16.0, 4e-6), (16.0, 40.0, 6e-6)]


def check_products(name, got, ref, dtype, tol):
    got, ref = to_np(got), np.asarray(ref)
    off = np.abs(got - ref) / np.abs(ref) - HALF_STEP[dtype] * (1 + 1e-5) - tol
    print("%s worst relative excess %.2e" % (name, off.max()), flush=True)
    assert np.all(np.abs(ref) > 1e-30) and np.all(off <= 0), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lo,hi,tol", FAR)
def test_gated_norm_slope_of_far_gates(dtype, lo, hi, tol):
    announce("gated norm, gates of %g to %g %s" % (lo, hi, dtype))
    for V in (64, 128, 256):
        o, dy = randn(90, dtype, 40, 3, V) + 3.0, randn(91, dtype, 40, 3, V) + 3.0
        g, w = far_gates(92, dtype, lo, hi, 40, 3, V), torch.linspace(0.5, 1.5, V, device="cuda")
        o, dy = torch.where(o.abs() < 1e-3, 1.0, o), torch.where(dy.abs() < 1e-3, 1.0, dy)
        want = layer_ref.gated_norm(o, g, w, dy)[2]
        check_products("dgate", gated_norm_backward(o, g, w, dy)[1], want, dtype, tol)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["token", "channel"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("lo,hi,tol", FAR)
def test_block_norm_slope_of_far_gates(dtype, gate, post, lo, hi, tol):
    announce("block norm, gates of %g to %g %s %s post %s" % (lo, hi, dtype, gate, post))
    for D in (264, 2056):
        x, y, wp, wq, _, dxo, _ = block_inputs(dtype, 40, D, "none", post, 93)
        y, dxo = (torch.where(t.abs() < 1e-3, 1.0, t) for t in (y, dxo))
        g = far_gates(99, dtype, lo, hi, *((40,) if gate == "token" else (40, D)))
        wq = None if wq is None else torch.linspace(0.5, 1.5, D, device="cuda")
        if gate == "token":  # terms of one sign, whose sum is of their size
            y, dxo = y.abs(), dxo.abs()
        want = layer_ref.block_norm(x, y, wp, wq, g, 0.3, dx_out=dxo, dh=np.zeros(x.shape))["dgate"]
        got = block_norm_backward(x, y, wp, dxo, None, w_post=wq, raw_gate=g, residual_scale=0.3)[4]
        check_products("dgate", got, want, dtype, tol)


# ------------------------------------------------------------------ several tokens per block


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,D", [(2100, 2048), (700, 8192), (9000, 72)])
def test_block_norm_with_several_tokens_per_block(dtype, gate, post, T, D):
    # the backward's blocks: 1024, 256 and 4096, so each takes two or three tokens
    announce("block norm %s gate %s post %s T%d D%d" % (dtype, gate, post, T, D))
    block_check(dtype, *block_inputs(dtype, T, D, gate, post, 110))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "channel"])
def test_post_norm_weights_of_rows_larger_than_the_caches(dtype, gate):
    announce("block norm past the caches, dw_post %s %s" % (dtype, gate))
    T, D = (12000 if dtype is BF16 else 6000), 4096
    x, y, wp, wq, gt, dxo, dh = block_inputs(dtype, T, D, gate, True, 120)
    kw = dict(w_post=wq, residual_scale=0.4)
    got = block_norm_backward(x, y, wp, dxo, dh, raw_gate=gt, **kw)
    sums = [torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(2)]
    for a in range(0, T, 500):  # one token per block
        s = slice(a, min(a + 500, T))
        part = block_norm_backward(x[s], y[s], wp, dxo[s], dh[s], raw_gate=None if gt is None else gt[s], **kw)
        for total, p in zip(sums, part[2:4]):
            total += p.double()
    assert rel(to_np(got[2]), to_np(sums[0])) <= 1e-5 and rel(to_np(got[3]), to_np(sums[1])) <= 1e-5
