"""GPU parity of the group norm, forward and backward, against the FP64
reference (needs an MI355X).

Tolerances. As for the gated and block norms: every output is fp32 arithmetic
rounded once, half a step of the dtype per element plus the fp32 error of the
terms it is formed from, 4e-6 of them and of their root mean square over the
row (sums of at most 8192 terms in a tree of serial runs of 16 and 13 levels,
29 roundings of 2^-24, and about 12 more of the factors). The terms of a
centred value n are r (|z| + |mean|), those of a gradient the products that it
is the difference of; the reference returns their sizes. Parameter gradients
are fp32 sums over rows: normalised L2 1e-5.
"""
import numpy as np
import pytest
import torch

from oracle import ssm_ref
from recompute_kda_chunked_amd import group_norm, group_norm_backward, group_norm_forward, ssm
from test_gpu_norms import check, randn
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
KINDS = [("none", "silu"), ("none", "sigmoid"), ("none", "none"), ("after", "silu"), ("after", "sigmoid"),
         ("first", "silu"), ("first", "sigmoid")]


def options(gate, act, groups, center, eps=1e-6):
    return dict(groups=groups, eps=eps, activation=act, center=center, gate_first=gate == "first")


def parity(dtype, T, groups, W, gate, act, center, bias, seed=1, shift=0.1, scale=1.5, far=False):
    C = groups * W
    x, dy = randn(seed, dtype, T, C, scale=scale, shift=shift), randn(seed + 1, dtype, T, C)
    g = None if gate == "none" else randn(seed + 2, dtype, T, C, scale=2.0)
    w = randn(seed + 3, F32, C, scale=0.3, shift=1.0)
    b = randn(seed + 4, F32, C, scale=0.3) if bias else None
    kw = options(gate, act, groups, center)
    ref = ssm_ref.group_norm(x, w, b, g, dy=dy, **kw)
    pt = ref["tz"] * np.abs(to_np(w)) + (np.abs(to_np(b)) if bias else 0.0)  # the terms of p
    if gate == "after":
        pt = pt * np.abs(ssm_ref._act(act, to_np(g))[0])
    check("y", group_norm_forward(x, w, b, g, **kw), ref["y"], dtype, terms=pt + np.abs(ref["y"]))
    dx, dw, db, dg = group_norm_backward(x, w, b, g, dy, **kw)
    check("dx", dx, ref["dx"], dtype, terms=ref["tdx"])
    assert (db is None) == (b is None) and (dg is None) == (g is None)
    if g is not None:
        check("dgate", dg, ref["dgate"], dtype, terms=ref["tdgate"])
    # of values far from zero each n carries its mean's roundings, 4e-6 of its terms as above,
    # so a channel's sum is within 4e-6 of the sum of its rows' |dp| r (|z| + |mean|)
    extra = 4e-6 * np.linalg.norm(np.sum(ref["tdw"], 0)) / np.linalg.norm(ref["dw"]) if far else 0.0
    assert dw.dtype is F32 and rel(to_np(dw), ref["dw"]) <= 1e-5 + extra
    if bias:
        assert rel(to_np(db), ref["db"]) <= 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,act", KINDS)
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("T,groups,W", [(1, 1, 64), (5, 3, 72), (67, 12, 200), (2, 2, 1160)])
def test_group_norm(dtype, gate, act, center, T, groups, W):
    announce("group norm %s %s %s center %s T%d %dx%d" % (dtype, gate, act, center, T, groups, W))
    parity(dtype, T, groups, W, gate, act, center, bias=center)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,groups,W", [(3, 1, 8), (40, 130, 8), (9, 33, 16), (131, 7, 32), (3, 1, 8192), (600, 5, 512),
                                        (7, 2, 520), (33, 2, 1024), (5, 1, 1032), (1000, 64, 64), (3, 3, 4104)])
def test_group_norm_widths(dtype, T, groups, W):
    announce("group norm widths %s T%d %dx%d" % (dtype, T, groups, W))
    for gate, center, bias in (("none", True, False), ("after", False, True), ("first", True, True)):
        parity(dtype, T, groups, W, gate, "silu", center, bias, seed=11)


@pytest.mark.parametrize("gate", ["none", "after", "first"])
def test_group_norm_of_groups_far_from_zero(gate):
    announce("group norm of values around 300, %s" % gate)
    parity(F32, 37, 6, 96, gate, "sigmoid", True, True, seed=21, shift=300.0, far=True)


def test_group_norm_zero_tiny_and_large_rows():
    announce("group norm, rows of zeros, of one value, tiny and large")
    x = randn(31, F32, 6, 128)
    x[0], x[1], x[2], x[3] = 0.0, 5.0, x[2] * 1e-20, x[3] * 1e15
    g, dy, w, b = randn(32, F32, 6, 128, scale=40.0), randn(33, F32, 6, 128), randn(34, F32, 128), randn(35, F32, 128)
    for gate in (None, g):
        kw = dict(groups=4, activation="silu")
        ref = ssm_ref.group_norm(x, w, b, gate, dy=dy, **kw)
        y, got = group_norm_forward(x, w, b, gate, **kw), group_norm_backward(x, w, b, gate, dy, **kw)
        for name, a, r in zip(("y", "dx", "dw", "db"), (y, *got), (ref["y"], ref["dx"], ref["dw"], ref["db"])):
            assert np.isfinite(to_np(a)).all() and rel(to_np(a), r) <= 1e-5, name
        for i in range(6):  # each row by itself: their gradients differ by 10^20
            assert rel(to_np(y[i]), ref["y"][i]) <= 1e-5 and rel(to_np(got[0][i]), ref["dx"][i]) <= 1e-5, i


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
def test_group_norm_slices_and_autograd(dtype, gate):
    announce("group norm of slices of wider rows, %s %s" % (dtype, gate))
    T, C = 33, 240
    wide = torch.full((T, 3 * C + 16), float("nan"), dtype=dtype, device="cuda")
    x, g = wide[:, 8:8 + C], wide[:, 2 * C:3 * C]
    x.copy_(randn(41, dtype, T, C))
    g.copy_(randn(42, dtype, T, C))
    w, b = randn(43, F32, C), randn(44, F32, C)
    kw = options(gate, "silu", 3, True)
    gg = None if gate == "none" else g
    leaves = [t.detach().requires_grad_(True) for t in (x, w, b, gg) if t is not None]
    y = group_norm(*leaves, **kw)
    dy = randn(45, dtype, C, T).t()  # not contiguous
    got = torch.autograd.grad(y, leaves, dy)
    plain = [None if t is None else t.contiguous() for t in (x, w, b, gg)]
    want = group_norm_backward(*plain, dy.contiguous(), **kw)
    again = group_norm_backward(*plain, dy.contiguous(), **kw)
    assert torch.equal(y, group_norm_forward(*plain, **kw))
    for a, r, s in zip(got, [t for t in want if t is not None], [t for t in again if t is not None]):
        assert torch.equal(a, r) and torch.equal(r, s)
    with torch.no_grad():  # further leading dimensions
        assert torch.equal(group_norm(*[t.view(3, 11, C) if t is not None and t.dim() == 2 else t for t in plain],
                                      **kw).view(T, C), y)


def test_group_norm_no_rows_and_one_graph():
    announce("group norm of no rows; captured and replayed")
    w, b = randn(51, F32, 64), randn(52, F32, 64)
    none = torch.empty(0, 64, device="cuda")
    assert group_norm(none, w, b, groups=2).shape == (0, 64)
    dx, dw, db, dg = group_norm_backward(none, w, b, None, none, groups=2)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all()) and dg is None
    x, g, dy = (randn(s, BF16, 70, 512) for s in (53, 54, 55))
    w, b = randn(56, F32, 512), randn(57, F32, 512)
    kw = dict(groups=8, gate_first=True)

    def both():
        return (group_norm_forward(x, w, b, g, **kw), *group_norm_backward(x, w, b, g, dy, **kw))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for s in (61, 62, 63):
        x.copy_(randn(s, BF16, 70, 512))
        dy.copy_(randn(s + 10, BF16, 70, 512))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, r) for a, r in zip(out, want))


def test_group_norm_past_32_bits():
    announce("group norm past 2^31 elements")
    T, C = 1_050_000, 2048 + 64
    x = torch.empty(T, C, dtype=BF16, device="cuda")
    x[:1000] = randn(71, BF16, 1000, C)
    x[1000:-1000] = 1.0
    x[-1000:] = x[:1000]
    w = randn(72, F32, C)
    y = group_norm_forward(x, w, groups=4, activation="none")
    assert torch.equal(y[-1000:], group_norm_forward(x[-1000:].clone(), w, groups=4, activation="none"))
    assert torch.equal(y[:1000], y[-1000:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("T", [0, 1, 300])
def test_gradients_of_parameters_that_are_not_given(dtype, gate, T):
    announce("dbias without a bias, a bias without dbias %s %s T%d" % (dtype, gate, T))
    x, dy = randn(81, dtype, T, 144), randn(82, dtype, T, 144)
    g, w, zero = None if gate == "none" else randn(83, dtype, T, 144), randn(84, F32, 144), torch.zeros(144, device="cuda")
    kw = options(gate, "silu", 2, True)

    def call(bias, dbias):
        dev, p = ssm._group_norm_problem(x, w, bias, g, 2, 1e-6, "silu", True, gate == "first", dy)
        out = [torch.full_like(t, float("nan")) for t in (x, x if g is None else g, w)]
        ssm._call(dev, "kda_group_norm_bwd", p, x, g, w, bias, dy, out[0], None if g is None else out[1], out[2], dbias,
                  workspace=ssm._workspace(dev, "kda_group_norm_bwd", p))
        return [out[0], out[2]] + ([] if g is None else [out[1]])

    dx, dw, db, dg = group_norm_backward(x, w, zero, g, dy, **kw)
    want = [dx, dw] + ([] if g is None else [dg])
    got = torch.full_like(w, float("nan"))
    for bias, dbias in ((None, got), (zero, None), (None, None)):
        assert all(torch.equal(a, b) for a, b in zip(call(bias, dbias), want))
    assert torch.equal(got, db)
