"""GPU parity of the short convolution (forward, backward, decoding) against
the FP64 reference (needs an MI355X).

Tolerances. y and dx are fp32 sums of at most 5 products, with the sigmoid's
few roundings, rounded once to the dtype: half a step (2^-8 of the value for
bf16) plus 16 roundings of 2^-24, 1e-6, of the terms' magnitudes (2e-6
allowed; see magnitudes()). States are copies: exact. dweight and dbias are fp32 sums over
the tokens of terms with that error: normalised L2 1e-5.
"""
import numpy as np
import pytest
import torch

from oracle import layer_ref
from recompute_kda_chunked_amd import (short_conv, short_conv_backward, short_conv_forward,
                                       short_conv_update)
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def randn(seed, dtype, *shape, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def inputs(dtype, lens, C, W, seed=1, bias=True):
    T, N = sum(lens), len(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return dict(x=randn(seed, dtype, T, C), w=randn(seed + 1, F32, C, W, scale=0.6),
                b=randn(seed + 2, F32, C, scale=0.5) if bias else None,
                init=randn(seed + 3, dtype, N, W - 1, C), dy=randn(seed + 4, dtype, T, C),
                df=randn(seed + 5, dtype, N, W - 1, C), cu=cu,
                cud=torch.tensor(cu, dtype=torch.int32, device="cuda"))


def near(name, got, ref, mag, dtype):
    got = to_np(got)
    off = np.abs(got - ref) - HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-5) - 2e-6 * mag
    print("%s worst excess %.2e" % (name, off.max() if off.size else 0), flush=True)
    assert np.isfinite(got).all() and np.all(off <= 0), name


def magnitudes(x, w, b, init, cu, dy, df):
    """Sums of the magnitudes of the terms of p (the activation's argument),
    and of dx and the initial state's gradient. A term of those is dy act'(p)
    w: act' (at most 1.1) adds its roundings and its slope (at most 0.5) times
    the error of p."""
    a = lambda t: None if t is None else np.abs(to_np(t))  # noqa: E731
    p = layer_ref.short_conv(a(x), a(w), a(b), cu, a(init), "none")["y"]
    f = layer_ref.short_conv(a(x), a(w), a(b), cu, a(init), "none", a(dy) * (1.1 + 0.5 * p), a(df))
    return p, f["dx"], f["dinit"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens,C", [([1], 8), ([5, 0, 1, 2, 9, 0], 72), ([0, 0, 3], 8),
                                    ([200, 1, 3, 130], 264), ([63, 64, 65, 2], 520), ([333], 1032)])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_forward_and_backward(dtype, W, lens, C, act):
    announce("short conv %s W%d %s C%d %s" % (dtype, W, lens, C, act))
    for bias, states in ((True, True), (False, False)):
        v = inputs(dtype, lens, C, W, bias=bias)
        init, df = (v["init"], v["df"]) if states else (None, None)
        ref = layer_ref.short_conv(v["x"], v["w"], v["b"], v["cu"], init, act, v["dy"], df)
        my, mdx, mdi = magnitudes(v["x"], v["w"], v["b"], init, v["cu"], v["dy"], df)
        y, final = short_conv_forward(v["x"], v["w"], v["b"], v["cud"], initial_state=init,
                                      output_final_state=True, activation=act)
        near("y", y, ref["y"], my, dtype)
        assert np.array_equal(to_np(final), ref["final"])
        dx, dw, db, di = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], initial_state=init,
                                             d_final_state=df, activation=act)
        near("dx", dx, ref["dx"], mdx, dtype)
        assert rel(to_np(dw), ref["dweight"]) <= 1e-5
        assert db is None if v["b"] is None else rel(to_np(db), ref["dbias"]) <= 1e-5
        if states:
            near("dinit", di, ref["dinit"], mdi, dtype)
        else:
            assert di is None


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_sequence_without_cu_seqlens(dtype):
    announce("short conv without cu_seqlens %s" % dtype)
    v = inputs(dtype, [77], 40, 4, seed=10)
    kw = dict(initial_state=v["init"])
    assert torch.equal(short_conv_forward(v["x"], v["w"], v["b"], **kw),
                       short_conv_forward(v["x"], v["w"], v["b"], v["cud"], **kw))
    a = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], **kw)
    b = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], **kw)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_many_short_sequences_and_long_runs():
    announce("300 sequences; 20000 tokens")
    gen = np.random.default_rng(3)
    for lens, C in ((list(gen.integers(0, 9, 300)), 64), ([20000, 7, 500], 64)):
        lens = [int(n) for n in lens]
        v = inputs(BF16, lens, C, 4, seed=20)
        ref = layer_ref.short_conv(v["x"], v["w"], v["b"], v["cu"], v["init"], "silu", v["dy"], v["df"])
        my, mdx, mdi = magnitudes(v["x"], v["w"], v["b"], v["init"], v["cu"], v["dy"], v["df"])
        y, final = short_conv_forward(v["x"], v["w"], v["b"], v["cud"], initial_state=v["init"],
                                      output_final_state=True)
        got = [short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], initial_state=v["init"],
                                   d_final_state=v["df"]) for _ in range(2)]
        near("y", y, ref["y"], my, BF16)
        near("dx", got[0][0], ref["dx"], mdx, BF16)
        near("dinit", got[0][3], ref["dinit"], mdi, BF16)
        assert np.array_equal(to_np(final), ref["final"])
        assert rel(to_np(got[0][1]), ref["dweight"]) <= 1e-5 and rel(to_np(got[0][2]), ref["dbias"]) <= 1e-5
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_rows_of_no_sequence_are_zero():
    announce("rows behind the last sequence")
    v = inputs(BF16, [5, 6, 9], 64, 4, seed=30)
    cu = torch.tensor([0, 5, 11], dtype=torch.int32, device="cuda")
    init, df = v["init"][:2], v["df"][:2]
    y, final = short_conv_forward(v["x"], v["w"], v["b"], cu, initial_state=init, output_final_state=True)
    dx, dw, db, di = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], cu, initial_state=init, d_final_state=df)
    part = (v["x"][:11], v["w"], v["b"])
    y2, final2 = short_conv_forward(*part, cu, initial_state=init, output_final_state=True)
    want = short_conv_backward(*part, v["dy"][:11], cu, initial_state=init, d_final_state=df)
    assert torch.equal(y[:11], y2) and torch.equal(final, final2) and bool((y[11:] == 0).all())
    assert torch.equal(dx[:11], want[0]) and bool((dx[11:] == 0).all())
    assert torch.equal(di, want[3]) and rel(to_np(dw), to_np(want[1])) <= 1e-6
    # no sequence at all, and bounds outside the tokens
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert bool((short_conv_forward(*part, none) == 0).all())
    wild = torch.tensor([-3, 5, 10 ** 9], dtype=torch.int32, device="cuda")
    assert torch.equal(short_conv_forward(*part, wild, initial_state=init), y2)
    late = torch.tensor([3, 11], dtype=torch.int32, device="cuda")  # tokens before the first sequence
    y3 = short_conv_forward(*part, late, initial_state=init[:1])
    assert bool((y3[:3] == 0).all())
    assert torch.equal(y3[3:], short_conv_forward(v["x"][3:11].clone(), v["w"], v["b"], initial_state=init[:1]))
    dx3 = short_conv_backward(*part, v["dy"][:11], late, initial_state=init[:1])[0]
    assert bool((dx3[:3] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(dtype):
    announce("short conv autograd %s" % dtype)
    v = inputs(dtype, [30, 2, 18], 64, 3, seed=40)
    leaves = [v["x"], v["w"], v["b"], v["init"]]
    want = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], initial_state=v["init"],
                               d_final_state=v["df"])
    for t in leaves:
        t.requires_grad_(True)
    y, final = short_conv(v["x"], v["w"], v["b"], v["cud"], initial_state=v["init"], output_final_state=True)
    torch.autograd.backward((y, final), (v["dy"], v["df"]))
    for t, g in zip(leaves, want):
        assert torch.equal(t.grad, g)
    for t in leaves:
        t.grad = None
    short_conv(v["x"], v["w"], v["b"], v["cud"], initial_state=v["init"], output_final_state=True)[1].backward(v["df"])
    with torch.no_grad():
        zero = short_conv_backward(v["x"], v["w"], v["b"], torch.zeros_like(v["dy"]), v["cud"],
                                   initial_state=v["init"], d_final_state=v["df"])
    for t, g in zip(leaves, zero):
        assert torch.equal(t.grad, g)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [1] * 7, [3, 0, 1, 6, 2]])
def test_update(dtype, W, lens):
    announce("short conv update %s W%d %s" % (dtype, W, lens))
    for C in (8, 328):
        v = inputs(dtype, lens, C, W, seed=50)
        pool = randn(60, dtype, len(lens) + 3, W - 1, C)
        idx = torch.randperm(len(lens) + 3, generator=torch.Generator().manual_seed(1))[:len(lens)]
        idx = idx.to(torch.int32).cuda()
        start = pool.clone()
        ref = layer_ref.short_conv(v["x"], v["w"], v["b"], v["cu"], start[idx.long()])
        my = magnitudes(v["x"], v["w"], v["b"], start[idx.long()], v["cu"], v["dy"], v["df"])[0]
        for one in ([False, True] if lens == [1] * len(lens) else [False]):
            pool.copy_(start)
            y = short_conv_update(v["x"], v["w"], v["b"], pool, None if one else v["cud"], state_indices=idx)
            near("y", y, ref["y"], my, dtype)
            want = start.clone()
            want[idx.long()] = torch.tensor(ref["final"], device="cuda").to(dtype)
            assert torch.equal(pool, want)


def test_update_padding_strides_and_rows_behind():
    announce("short conv update, padding and strides")
    C = 64
    v = inputs(BF16, [2, 1, 1, 2], C, 4, seed=70)
    wide = torch.full((6, 3 * C), float("nan"), dtype=BF16, device="cuda")
    wide[:, C:2 * C] = v["x"]
    x = wide[:, C:2 * C]
    cu = torch.tensor([0, 2, 3, 4, 4], dtype=torch.int32, device="cuda")
    idx = torch.tensor([1, -1, 9, 0], dtype=torch.int32, device="cuda")  # 9: past the pool
    pool = randn(71, BF16, 2, 3, C)
    start = pool.clone()
    out = torch.full((6, C), 5.0, dtype=BF16, device="cuda")
    short_conv_update(x, v["w"], v["b"], pool, cu, state_indices=idx, out=out)
    ref = layer_ref.short_conv(v["x"][:2], v["w"], v["b"], [0, 2], start[1:2])
    assert rel(to_np(out[:2]), ref["y"]) <= 2.0 ** -8
    assert bool((out[2] == 0).all()) and bool(torch.isnan(out[3]).all()) and bool((out[4:] == 5).all())
    assert np.array_equal(to_np(pool[1]), ref["final"][0]) and torch.equal(pool[0], start[0])
    assert torch.equal(short_conv_forward(x, v["w"], v["b"], v["cud"]),
                       short_conv_forward(v["x"], v["w"], v["b"], v["cud"]))
    a = short_conv_backward(x, v["w"], v["b"], v["dy"], v["cud"])
    b = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"])
    assert all(torch.equal(s, t) for s, t in zip(a[:3], b[:3]))


def test_update_of_a_slot_named_twice():
    announce("short conv update, a slot named twice")
    for C in (8, 2056):
        v = inputs(F32, [1, 0, 1, 1], C, 3, seed=75)
        pool = randn(76, F32, 3, 2, C)
        idx = torch.tensor([2, 1, 1, 2], dtype=torch.int32, device="cuda")
        other, pad = pool.clone(), torch.tensor([2, 1, 1, -1], dtype=torch.int32, device="cuda")
        got = short_conv_update(v["x"], v["w"], v["b"], pool, v["cud"], state_indices=idx)
        want = short_conv_update(v["x"], v["w"], v["b"], other, v["cud"], state_indices=pad)
        assert torch.equal(got[:2], want[:2]) and bool(torch.isnan(got[2]).all()) and torch.equal(pool, other)


def test_update_continues_forward():
    announce("convolution: prompt, then tokens")
    v = inputs(F32, [40, 25], 96, 4, seed=80)
    whole, final = short_conv_forward(v["x"], v["w"], v["b"], v["cud"], output_final_state=True)
    cut = [37, 22]
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(v["cu"], cut)]).cuda()
    pcu = torch.tensor([0, 37, 59], dtype=torch.int32, device="cuda")
    _, state = short_conv_forward(v["x"][rows], v["w"], v["b"], pcu, output_final_state=True)
    for j in range(3):
        at = torch.tensor([a + n + j for a, n in zip(v["cu"], cut)], device="cuda")
        assert torch.equal(short_conv_update(v["x"][at], v["w"], v["b"], state), whole[at])
    assert torch.equal(state, final)


def test_no_tokens():
    announce("convolution of no tokens")
    v = inputs(BF16, [4, 2], 64, 4, seed=90)
    x, cu = v["x"][:0], torch.zeros(3, dtype=torch.int32, device="cuda")
    y, final = short_conv_forward(x, v["w"], v["b"], cu, initial_state=v["init"], output_final_state=True)
    assert y.shape == (0, 64) and torch.equal(final, v["init"])
    dx, dw, db, di = short_conv_backward(x, v["w"], v["b"], x, cu, initial_state=v["init"], d_final_state=v["df"])
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all()) and torch.equal(di, v["df"])
    assert short_conv_update(x, v["w"], v["b"], v["init"].clone(), cu).shape == (0, 64)


def test_captured_and_replayed():
    announce("convolution in a graph")
    v = inputs(BF16, [100, 60, 40], 512, 4, seed=100)
    pool = randn(101, BF16, 4, 3, 512)
    one = randn(102, BF16, 3, 512)

    def step(pool):
        return (*short_conv_forward(v["x"], v["w"], v["b"], v["cud"], initial_state=v["init"], output_final_state=True),
                *short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], initial_state=v["init"],
                                     d_final_state=v["df"]),
                short_conv_update(one, v["w"], v["b"], pool))

    other = pool.clone()
    graph = torch.cuda.CUDAGraph()
    step(pool.clone())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(pool)
    for k in range(3):
        v["x"].mul_(0.5)
        one.add_(0.25)
        if k == 1:
            v["cud"].copy_(torch.tensor([0, 0, 130, 200], dtype=torch.int32))
        want = step(other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(pool, other), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_rows_larger_than_the_caches(dtype, W):
    announce("convolution past the caches %s W%d" % (dtype, W))  # 600 MB and more per launch
    C, each = 4096, 5000 if dtype is F32 else 10001
    v = inputs(dtype, [each, 0, 3, 2 * each - 3, each], C, W, seed=110)
    y, final = short_conv_forward(v["x"], v["w"], v["b"], v["cud"], initial_state=v["init"], output_final_state=True)
    got = short_conv_backward(v["x"], v["w"], v["b"], v["dy"], v["cud"], initial_state=v["init"], d_final_state=v["df"])
    for c in range(0, C, 512):  # the same channels in smaller launches
        s = slice(c, c + 512)
        part = {k: v[k][..., s].contiguous() for k in ("x", "b", "init", "dy", "df")}
        w = v["w"][s]
        a = short_conv_forward(part["x"], w, part["b"], v["cud"], initial_state=part["init"], output_final_state=True)
        assert torch.equal(y[:, s], a[0]) and torch.equal(final[..., s], a[1])
        b = short_conv_backward(part["x"], w, part["b"], part["dy"], v["cud"], initial_state=part["init"],
                                d_final_state=part["df"])
        assert torch.equal(got[0][:, s], b[0]) and torch.equal(got[3][..., s], b[3])
        assert rel(to_np(got[1][s]), to_np(b[1])) <= 1e-5 and rel(to_np(got[2][s]), to_np(b[2])) <= 1e-5


def test_update_of_sequences_that_clamping_leaves_empty():
    announce("short conv update, a sequence before the first token names the slot of the next")
    v = inputs(F32, [3], 64, 4, seed=120)
    pool, idx = randn(121, F32, 2, 3, 64), torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    other = pool.clone()
    cu = torch.tensor([-4, -2, 3], dtype=torch.int32, device="cuda")
    got = short_conv_update(v["x"], v["w"], v["b"], pool, cu, state_indices=idx)
    assert torch.equal(got, short_conv_update(v["x"], v["w"], v["b"], other, v["cud"], state_indices=idx[:1]))
    assert torch.equal(pool, other)


@pytest.mark.parametrize("n,C", [(1026, 8), (3000, 1032)])
def test_update_of_slots_named_twice_among_many(n, C):
    announce("short conv update, slots named twice among %d sequences" % n)
    v = inputs(F32, [1] * n, C, 3, seed=130)
    pool = randn(131, F32, n + 1, 2, C)
    other = pool.clone()
    idx = torch.randperm(n + 1, generator=torch.Generator().manual_seed(2))[:n].to(torch.int32).cuda()
    pad, bad = idx.clone(), torch.zeros(n, dtype=torch.bool, device="cuda")
    for i, j in ((1025, 1024), (n - 1, 0), (700, 699)):
        idx[i], pad[i], bad[i] = idx[j], -1, True
    got = short_conv_update(v["x"], v["w"], v["b"], pool, state_indices=idx)
    want = short_conv_update(v["x"], v["w"], v["b"], other, state_indices=pad)
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[~bad]) and torch.equal(pool, other)


def test_update_of_many_sequences_without_indices():
    announce("70000 sequences without indices")
    v = inputs(F32, [1] * 70000, 8, 2, seed=140)
    pool = v["init"].clone()
    y = short_conv_update(v["x"], v["w"], v["b"], pool)
    some = slice(65530, 65550)
    ref = layer_ref.short_conv(v["x"][some], v["w"], v["b"], range(21), v["init"][some])
    assert rel(to_np(y[some]), ref["y"]) <= 1e-6 and torch.equal(pool[:, 0], v["x"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [8, 2056])
def test_update_zeroes_new_rows_of_no_sequence(dtype, C):
    announce("short conv update, rows of no sequence in a new y %s C%d" % (dtype, C))
    v = inputs(dtype, [5, 6, 7, 5], C, 4, seed=150)
    pool, start = randn(151, dtype, 4, 3, C), randn(151, dtype, 4, 3, C)
    cud = torch.empty(5, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    cud.copy_(v["cud"])
    short_conv_update(v["x"], v["w"], v["b"], pool.clone(), cud)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = short_conv_update(v["x"], v["w"], v["b"], pool, cud)
    for cu in ([0, 5, 11, 18, 23], [0, 2, 3, 3, 5], [1, 2, 2, 4, 4], [0] * 5, [23] * 5):
        cud.copy_(torch.tensor(cu, dtype=torch.int32))
        pool.copy_(start)
        a, b = start.clone(), start.clone()
        kept = short_conv_update(v["x"], v["w"], v["b"], a, cud, out=torch.full_like(v["x"], 7.0))
        for _ in range(3):
            torch.full_like(v["x"], float("nan"))
        got = short_conv_update(v["x"], v["w"], v["b"], b, cud)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((kept[:cu[0]] == 7).all()) and bool((kept[cu[-1]:] == 7).all())
        assert bool((got[:cu[0]] == 0).all()) and bool((got[cu[-1]:] == 0).all())
        assert torch.equal(got[cu[0]:cu[-1]], kept[cu[0]:cu[-1]]) and torch.equal(out, got)
        assert torch.equal(a, b) and torch.equal(a, pool)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert bool((short_conv_update(v["x"], v["w"], v["b"], start, none) == 0).all())


def test_update_zeroes_many_new_rows():
    announce("short conv update, 110 MB of rows that belong to no sequence")
    T, C = 7000, 4096
    x, w, pool = randn(160, F32, T, C), randn(161, F32, C, 4), randn(162, F32, 3, 3, C)
    for cu in ([0, 2, 2, 5], [6900, 6902, 6902, 6905], [3000, 3002, 3002, 3005]):
        torch.full_like(x, float("nan"))
        got = short_conv_update(x, w, None, pool, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert bool((got[:cu[0]] == 0).all()) and bool((got[cu[-1]:] == 0).all())
        assert bool((got[cu[0]:cu[-1]] != 0).any(1).all())
