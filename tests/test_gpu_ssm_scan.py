"""GPU parity of the selective scan, forward and backward, against the FP64
reference (needs an MI355X).

Tolerances. Decays and step sizes are positive, so the reference run on the
inputs' absolute values gives the sum of the sizes of the terms of every
output, and each element is held to its own:
  y, dx, dB, dC   half a step of the dtype of the value, plus of the terms: in
                  bf16 one rounding of a score or a state, 2^-8, and 1e-5 for
                  fp32's roundings (sums of at most 128 + 128 terms in serial
                  runs of 32, the scores, decays and step sizes: below 100
                  roundings of 2^-24 = 6e-6); in fp32 1e-5
  draw_dt         half a step, plus 1e-5 of the terms of its chunk, over which
                  the decay's gradient is summed up and differs
  dA_log          (fp32) 1e-5 of its terms, and 1e-6 (16 roundings of 2^-24) of
                  those of a tile of 16 tokens, of which it takes differences
  states and their gradients, ddt_bias, dD  (fp32) 1e-5 of their terms
In bf16 the fp32 outputs come from exact products too: a weighted row or state is
three bf16, of 8 bits each, which leaves 2^-25 of it.
"""
import numpy as np
import pytest
import torch

from oracle import ssm_ref
from recompute_kda_chunked_amd import (group_norm, short_conv, short_conv_update, ssm_recurrent, ssm_scan,
                                       ssm_scan_backward, ssm_scan_forward)
from test_gpu_recurrent import leave_nan
from test_gpu_ssm_recurrent import ssm_inputs
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
NAMES = ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias")


def make(lens, H, G, N, P, dtype, seed, init=True, fused=False, **kw):
    x = dict(ssm_inputs(lens, H, G, N, P, dtype, seed, fused=fused, pool=False), **kw)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000)
    n = len(lens)
    x["init"] = torch.randn((n, H, N, P), generator=gen, device="cuda") if init else None
    x["dy"] = torch.randn(x["x"].shape, generator=gen, device="cuda").to(dtype)
    x["dfinal"] = torch.randn((n, H, N, P), generator=gen, device="cuda") if init else None
    return x


def forward(x, **kw):
    return ssm_scan_forward(*[x[k] for k in NAMES], x["cu"], initial_state=x["init"], dt_limit=x["limit"],
                            output_final_state=True, **kw)


def backward(x):
    return ssm_scan_backward(*[x[k] for k in NAMES], x["dy"], x["cu"], initial_state=x["init"],
                             d_final_state=x["dfinal"], dt_limit=x["limit"])


def reference(x, absolute=False):
    f = (lambda t: None if t is None else np.abs(to_np(t))) if absolute else (lambda t: None if t is None else to_np(t))
    args = [f(x[k]) if k in ("x", "B", "C", "D") else (None if x[k] is None else to_np(x[k])) for k in NAMES]
    return ssm_ref.scan(*args, x["cu_host"], f(x["init"]), limit=x["limit"], dy=f(x["dy"]), dfinal=f(x["dfinal"]))


def held(name, got, ref, bound):
    got, ref = to_np(got), np.asarray(ref)
    off = np.abs(got - ref) - bound - 2.0 ** -126  # below fp32's normal numbers: may be zero
    print("%s worst excess %.2e of %.2e, L2 %.2e" % (name, off.max() if off.size else 0, np.max(bound, initial=0), rel(got, ref)), flush=True)
    assert np.isfinite(got).all() and np.all(off <= 0), name


def chunk_sums(t, cu, Q):
    """Of each token, the sum over its chunk."""
    out = np.zeros_like(t)
    for a, b in zip(cu, cu[1:]):
        for s in range(a, b, Q):
            e = min(s + Q, b)
            out[s:e] = t[s:e].sum(0)
    return out


def parity(x):
    dtype = x["x"].dtype
    half, Q = HALF_STEP[dtype], 128 if dtype is BF16 else 64
    one, two = 1e-5 if dtype is F32 else 2.0 ** -8 + 1e-5, 1e-5
    state = 1e-5
    y_ref, s_ref, g = reference(x)
    y_abs, s_abs, t = reference(x, absolute=True)
    y, final = forward(x)
    held("y", y, y_ref, half * np.abs(y_ref) + one * y_abs)
    held("final", final, s_ref, state * s_abs)
    dx, ddt, dA, dB, dC, dD, dbias, dinit = backward(x)
    held("dx", dx, g["dx"], half * np.abs(g["dx"]) + one * t["dx"])
    held("dB", dB, g["dB"], half * np.abs(g["dB"]) + one * t["dB"])
    held("dC", dC, g["dC"], half * np.abs(g["dC"]) + one * t["dC"])
    # a token's decay collects its chunk's terms, weighted with its own slope; A_log's with its step
    dt, slope = ssm_ref.step_sizes(to_np(x["raw_dt"]), None if x["dt_bias"] is None else to_np(x["dt_bias"]), x["limit"])
    terms = chunk_sums(t["tall"], x["cu_host"], Q) * slope
    held("draw_dt", ddt, g["draw_dt"], half * np.abs(g["draw_dt"]) + two * terms)
    held("dA_log", dA, g["dA_log"], 1e-5 * np.abs(t["dA_log"]) + 1e-6 * np.sum(dt * chunk_sums(t["tall"], x["cu_host"], 16), 0))
    if x["D"] is not None:
        held("dD", dD, g["dD"], 1e-5 * t["dD"])
    if x["dt_bias"] is not None:
        held("ddt_bias", dbias, g["ddt_bias"], two * terms.sum(0))
    assert (dD is None) == (x["D"] is None) and (dbias is None) == (x["dt_bias"] is None)
    if x["init"] is not None:
        held("dinit", dinit, g["dinit"], state * t["dinit"])
    else:
        assert dinit is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,H,G", [([1], 1, 1), ([37], 4, 2), ([130, 0, 1, 64, 65], 2, 1)])
def test_scan(dtype, N, P, lens, H, G):
    announce("scan %s N%d P%d %s H%d G%d" % (dtype, N, P, lens, H, G))
    parity(make(lens, H, G, N, P, dtype, 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,H,G", [([300], 3, 1), ([63, 127, 128, 129, 0, 2], 6, 3), ([1] * 20, 5, 5), ([257, 64], 8, 1)])
def test_scan_lengths_and_groups(dtype, lens, H, G):
    announce("scan lengths %s %s H%d G%d" % (dtype, lens, H, G))
    parity(make(lens, H, G, 64, 64, dtype, 2))
    parity(make(lens, H, G, 64, 64, dtype, 3, init=False))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_limits_and_missing_parameters(dtype):
    announce("scan with limits, without D and bias %s" % dtype)
    parity(make([70, 5], 4, 2, 64, 64, dtype, 4, limit=(0.05, 0.11)))
    parity(make([70, 5], 4, 2, 64, 64, dtype, 5, D=None))
    parity(make([70, 5], 4, 2, 64, 64, dtype, 6, dt_bias=None))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_large_and_vanishing_steps(dtype):
    announce("scan with steps from 1e-30 to 90 %s" % dtype)
    x = make([150], 4, 1, 64, 64, dtype, 7)
    x["dt_bias"].zero_()
    x["raw_dt"][:, 0], x["raw_dt"][:, 1] = -70.0, 90.0  # nothing written; only the own token seen
    x["raw_dt"][::9, 2], x["raw_dt"][4::9, 3] = 60.0, -60.0
    parity(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_decays_that_leave_nothing(dtype):
    announce("scan with exp(A_log) up to fp32's largest %s" % dtype)
    x = make([150, 3], 4, 1, 64, 64, dtype, 17)
    x["A_log"].copy_(torch.tensor([87.5, 30.0, 8.0, -80.0]))  # nothing, nothing, little and all of a state is left
    parity(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_long_steps(dtype):
    announce("scan whose decays forget within a few tokens %s" % dtype)
    x = make([400, 128, 37], 4, 1, 128, 64, dtype, 22)
    x["A_log"].add_(1.5)
    x["dt_bias"].zero_()
    parity(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,H,G,P", [([1500, 0, 1, 1100, 399], 2, 1, 64), ([2111], 3, 3, 128), ([40, 2500, 60], 1, 1, 64)])
def test_long_sequences_in_segments(dtype, lens, H, G, P):
    announce("long sequences %s %s H%d P%d" % (lens, dtype, H, P))
    x = make(lens, H, G, 128, P, dtype, 18)
    x["A_log"][0] = -6.0  # a state that lasts over segments
    parity(x)
    parity(dict(x, init=None, dfinal=None))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_short_sequences(dtype):
    announce("600 short sequences, heads of a group together and apart %s" % dtype)
    lens = [1 + (7 * n) % 4 for n in range(600)]
    parity(make(lens, 6, 1, 64, 64, dtype, 19))


def test_segments_of_ragged_batches_replayed():
    announce("long sequences: rows of no sequence, other lengths in a captured call")
    x = make([1500, 0, 1, 1100, 399], 2, 1, 128, 64, BF16, 20)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (*forward(x), *backward(x))
    for cu in ([0, 1500, 1500, 1501, 2601, 3000], [700, 2900, 2900, 2900, 2901, 2950], [0, 600, 1200, 1800, 2400, 3000],
               [5, 5, 5, 5, 5, 3000], [0, 0, 0, 0, 0, 0], [0, 3000, 3000, 3000, 3000, 3000]):
        x["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        leave_nan(x["x"].shape, BF16)
        ref = (*forward(x), *backward(x))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, ref))
        for n, (a, b) in enumerate(zip(cu, cu[1:])):  # each sequence by itself
            part = dict(x, **{k: x[k][a:b].contiguous() for k in ("x", "raw_dt", "B", "C", "dy")}, cu=None,
                        init=x["init"][n:n + 1].contiguous(), dfinal=x["dfinal"][n:n + 1].contiguous())
            if b - a == 0:
                assert torch.equal(ref[1][n], x["init"][n]) and torch.equal(ref[-1][n], x["dfinal"][n])
                continue
            one = (*forward(part), *backward(part))
            for i in (0, 1, 2, 3, 5, 6, 9):  # states differ by the roundings of their segments
                got = ref[i][n:n + 1] if i in (1, 9) else ref[i][a:b]
                assert rel(to_np(got), to_np(one[i])) <= (1e-5 if i in (1, 9) else 2.0 ** -8), (cu, n, i)
        for i in (0, 2, 3, 5, 6):
            assert bool((ref[i][:cu[0]] == 0).all()) and bool((ref[i][cu[-1]:] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_a_number_stays_in_its_sequence_and_behind_its_token(dtype, value):
    announce("scan with %s in one sequence %s" % (value, dtype))
    x = make([130, 1500, 70, 1300], 2, 2, 64, 64, dtype, 23)
    want = (*forward(x), *backward(x))
    bad = dict(x, x=x["x"].clone(), B=x["B"].clone())
    bad["x"][130 + 700, 0] = value
    bad["B"][130 + 700, 1] = value
    got = (*forward(bad), *backward(bad))
    for i in (0, 2, 3, 5, 6):  # rows: the others' as they were
        assert torch.equal(got[i][:130], want[i][:130]) and torch.equal(got[i][1630:], want[i][1630:])
    for i in (1, 9):
        assert torch.equal(got[i][[0, 2, 3]], want[i][[0, 2, 3]]) and not bool(torch.isfinite(got[i][1]).all() and i == 1)
    # chunks before the token's (128 or 64 tokens) are untouched, outputs from it on are not finite
    assert torch.equal(got[0][130:130 + 640], want[0][130:130 + 640])
    assert not bool(torch.isfinite(got[0][130 + 700]).any())


def test_offsets_past_32_bits():
    announce("scan: offsets past 2^31 elements")
    H, G, N, P, T = 64, 1, 64, 128, 262144 + 300
    x = make([70], H, G, N, P, BF16, 21)
    far = dict(x, init=torch.zeros((2, H, N, P), device="cuda"), dfinal=torch.zeros((2, H, N, P), device="cuda"),
               cu=torch.tensor([0, T - 70, T], dtype=torch.int32, device="cuda"))
    for k in ("x", "raw_dt", "B", "C", "dy"):
        far[k] = torch.zeros((T, *x[k].shape[1:]), dtype=BF16, device="cuda")
        far[k][T - 70:] = x[k]
    for k in ("init", "dfinal"):
        far[k][1] = x[k][0]
    a, b = (*forward(x), *backward(x)), (*forward(far), *backward(far))
    assert b[0].numel() > 2 ** 31
    for i in (0, 2, 3):
        assert torch.equal(a[i], b[i][T - 70:]), i
    for i in (1, 9):
        assert torch.equal(a[i][0], b[i][1]), i
    for i in (5, 6):  # the heads add up in another division
        assert rel(to_np(b[i][T - 70:]), to_np(a[i])) <= 2.0 ** -8
    assert not bool(b[0][:1000].any()) and not bool(b[2][-1000 - 70:-70].any())


def make_single(dtype):
    x = make([200], 2, 1, 64, 64, dtype, 8)
    return x, dict(x, cu=None)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_without_cu_seqlens_and_of_slices(dtype):
    announce("scan without cu_seqlens; of slices of wider rows %s" % dtype)
    x, y = make_single(dtype)
    for a, b in zip((*forward(x), *backward(x)), (*forward(y), *backward(y))):
        assert torch.equal(a, b)
    x, y = (make([33, 140], 4, 2, 128, 64, dtype, 9, fused=f) for f in (False, True))
    assert not y["x"].is_contiguous()
    wide = torch.full((173, 12), float("nan"), dtype=dtype, device="cuda")
    wide[:, 3:7] = y["raw_dt"]
    y["raw_dt"] = wide[:, 3:7]
    for a, b in zip((*forward(x), *backward(x)), (*forward(y), *backward(y))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,G", [(2, 2), (6, 1)])
def test_rows_of_no_sequence(dtype, H, G):
    announce("scan: rows of no sequence, clamped cu_seqlens %s" % dtype)
    x = make([3, 140, 0, 60, 7], H, G, 64, 64, dtype, 10)  # the first and the last tokens in no sequence
    cu = [3, 143, 143, 203]
    x.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), cu_host=cu, init=x["init"][:3].contiguous(),
             dfinal=x["dfinal"][:3].contiguous())
    for name in ("x", "raw_dt", "B", "C", "dy"):
        x[name][:3] = x[name][203:] = float("nan")
    leave_nan(x["x"].shape, dtype)
    y, final = forward(x)
    got = backward(x)
    for t in (y, got[0], got[1], got[3], got[4]):
        assert bool((t[:3] == 0).all()) and bool((t[203:] == 0).all())
    part = dict(x, **{k: x[k][3:203].contiguous() for k in ("x", "raw_dt", "B", "C", "dy")}, cu=x["cu"] - 3)
    want = (*forward(part), *backward(part))
    for i, (a, b) in enumerate(zip((y, final, *got), want)):
        assert torch.equal(a[3:203] if a.shape[0] == 210 else a, b), i
    none = dict(x, cu=torch.zeros(1, dtype=torch.int32, device="cuda"), init=None, dfinal=None)
    leave_nan(x["x"].shape, dtype)
    y, final = forward(none)
    got = backward(none)
    assert final.shape[0] == 0
    for t in (y, *got[:7]):
        assert bool((t == 0).all())
    far = dict(part, cu=torch.tensor([-7, 140, 140, 100000], dtype=torch.int32, device="cuda"))
    for a, b in zip((*forward(far), *backward(far)), want):
        assert torch.equal(a, b)


def test_no_tokens():
    announce("scan of no tokens")
    x = make([0, 0], 2, 1, 64, 64, BF16, 11)
    y, final = forward(x)
    assert y.shape == (0, 2, 64) and torch.equal(final, x["init"])
    got = backward(x)
    assert torch.equal(got[-1], x["dfinal"])
    assert all(bool((got[i] == 0).all()) for i in (2, 5, 6)) and got[0].shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd_repeats_and_partial_gradients(dtype):
    announce("scan autograd %s" % dtype)
    x = make([40, 100], 4, 2, 64, 64, dtype, 12)
    want = backward(x)
    leaves = [x[k].detach().requires_grad_(True) for k in (*NAMES, "init")]
    y, final = ssm_scan(*leaves[:7], x["cu"], initial_state=leaves[7], output_final_state=True)
    wide = x["dy"].transpose(0, 1).contiguous().transpose(0, 1)  # not contiguous
    got = torch.autograd.grad((y, final), leaves, (wide, x["dfinal"]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    y, final = ssm_scan(*leaves[:7], x["cu"], initial_state=leaves[7], output_final_state=True)
    only = torch.autograd.grad(final, leaves, x["dfinal"], allow_unused=True)
    ref = backward(dict(x, dy=torch.zeros_like(x["dy"])))
    for a, b in zip(only, ref):
        assert torch.equal(a, b)
    y = ssm_scan(leaves[0], x["raw_dt"], x["A_log"], x["B"], x["C"], None, None, x["cu"])
    g, = torch.autograd.grad(y, leaves[0], x["dy"])
    assert torch.equal(g, backward(dict(x, D=None, dt_bias=None, init=None, dfinal=None))[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pieces_of_a_sequence_and_decoding_continue_it(dtype):
    announce("scan in pieces, then token by token %s" % dtype)
    x = make([300, 41], 4, 2, 128, 64, dtype, 13)
    y, final = forward(x)
    # rounding points move with the pieces' chunks: each is held to the reference
    y_ref, s_ref, _ = reference(x)
    y_abs, s_abs, _ = reference(x, absolute=True)
    one, state = 1e-5 if dtype is F32 else 2.0 ** -8 + 1e-5, 1e-5
    lens, at, pool, rows = [300, 41], [0, 300], x["init"], []
    got = np.zeros_like(y_ref)
    for cut in ([100, 20], [97, 19]):
        r = torch.cat([torch.arange(a, a + m) for a, m in zip(at, cut)]).cuda()
        part = dict(x, **{k: x[k][r].contiguous() for k in ("x", "raw_dt", "B", "C")}, init=pool,
                    cu=torch.tensor([0, cut[0], sum(cut)], dtype=torch.int32, device="cuda"))
        yp, pool = forward(part)
        got[r.cpu().numpy()] = to_np(yp)
        at = [a + m for a, m in zip(at, cut)]
        rows.append(r)
    r = torch.cat([torch.arange(at[0], 300), torch.arange(at[1], 341)]).cuda()
    cu = torch.tensor([0, 300 - at[0], len(r)], dtype=torch.int32, device="cuda")
    yp = ssm_recurrent(*[x[k][r].contiguous() if k in ("x", "raw_dt", "B", "C") else x[k] for k in NAMES], pool, cu)
    got[r.cpu().numpy()] = to_np(yp)
    off = np.abs(got - y_ref) - HALF_STEP[dtype] * np.abs(y_ref) - one * y_abs
    assert np.all(off <= 0)
    assert np.all(np.abs(to_np(pool) - s_ref) <= 2 * state * s_abs)


def test_streams_and_graph_replay():
    announce("scan on two streams; captured with other lengths and replayed")
    xs = [make([150, 30, 80], 4, 2, 128, 64, BF16, s) for s in (14, 15)]
    want = [(*forward(x), *backward(x)) for x in xs]
    torch.cuda.synchronize()
    got = []
    for x in xs:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append((*forward(x), *backward(x)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))
    x = xs[0]
    graphs, outs = [], []
    for _ in range(2):  # two graphs of the same call: each has its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*forward(x), *backward(x)))
        graphs.append(g)
    for cu in ([0, 150, 180, 260], [0, 10, 20, 30], [5, 5, 5, 260], [0, 0, 129, 258]):
        x["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        x["x"].mul_(0.5)
        ref = (*forward(x), *backward(x))
        for g, out in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(s, t) for s, t in zip(out, ref))


def test_a_layer_in_training_and_decoding():
    announce("convolution, scan and norm together")
    H, G, N, P, lens = 8, 2, 64, 64, [90, 1, 150]
    T, C, inner = sum(lens), H * P + 2 * G * N, H * P
    gen = torch.Generator(device="cuda").manual_seed(16)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    cu = torch.tensor([0, 90, 91, 241], dtype=torch.int32, device="cuda")
    wide = randn(T, inner + C + 8)
    par = dict(cw=randn(C, 4, scale=0.4), cb=randn(C, scale=0.2), A=torch.rand(H, generator=gen, device="cuda"),
               D=randn(H), tb=randn(H) - 2.5, w=1 + randn(inner, scale=0.2))

    def layer(wide, par, cu=None, pools=None):
        gate, xbc, dt = wide[:, :inner], wide[:, inner:inner + C], wide[:, inner + C:]
        if pools is None:
            xbc = short_conv(xbc, par["cw"], par["cb"], cu, output_final_state=cu is not None)
            xbc, conv_state = xbc
        else:
            xbc = short_conv_update(xbc, par["cw"], par["cb"], pools[0])
        x, B, Cm = xbc.split([inner, G * N, G * N], 1)
        args = (x.view(-1, H, P), dt, par["A"], B.view(-1, G, N), Cm.view(-1, G, N), par["D"], par["tb"])
        if pools is None:
            y, state = ssm_scan(*args, cu, output_final_state=True)
        else:
            y = ssm_recurrent(*args, pools[1])
        y = group_norm(y.reshape(-1, inner), par["w"], None, gate, groups=G, center=False, gate_first=True)
        return (y, conv_state, state) if pools is None else y

    # training: gradients against differences along random directions
    leaves = {k: v.clone().requires_grad_(True) for k, v in par.items()}
    wl = wide.clone().requires_grad_(True)
    dy = randn(T, inner)
    y, conv_state, state = layer(wl, leaves, cu)
    y.backward(dy)
    with torch.no_grad():
        for name, t in (("wide", wl), *leaves.items()):
            d = torch.randn(t.shape, generator=gen, device="cuda")
            h = 1e-2 * t.norm() / d.norm() / 10

            def at(s):
                moved = {k: (v + s * h * d if k == name else v) for k, v in par.items()}
                out = layer(wide + s * h * d if name == "wide" else wide, moved, cu)[0]
                return (out.double() * dy.double()).sum()

            num = float((8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h))  # fourth order
            ana = float((t.grad.double() * d.double()).sum())
            size = float((t.grad.double() * d.double()).abs().sum())
            print("layer d%s %.5e by differences %.5e" % (name, ana, num), flush=True)
            # differences: fp32 outputs' roundings over the step (4e-6 of the loss's terms / h) and h^4
            loss = float((y.detach().double() * dy.double()).norm())
            assert abs(num - ana) <= 1e-3 * max(abs(ana), size / 30) + 4e-6 * loss / float(h)
        # decoding continues the sequences
        more = randn(3, 4, wide.shape[1])
        pools = (conv_state, state)
        full = torch.cat([torch.cat([wide[a:b], more[i]]) for i, (a, b) in enumerate(zip([0, 90, 91], [90, 91, 241]))])
        want = layer(full, par, torch.tensor([0, 94, 99, 253], dtype=torch.int32, device="cuda"))
        for j in range(4):
            got = layer(more[:, j].contiguous(), par, pools=pools)
            assert rel(to_np(got), to_np(want[0][[90 + j, 95 + j, 249 + j]])) <= 1e-5
        assert rel(to_np(pools[1]), to_np(want[2])) <= 1e-5
        assert rel(to_np(pools[0]), to_np(want[1])) <= 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("N,P", [(64, 128), (128, 64)])
def test_what_is_not_a_number_reaches_no_output_before_its_token(dtype, value, N, P):
    announce("scan with %s: outputs that the formulas keep free of it %s N%d P%d" % (value, dtype, N, P))
    x = make([40, 300, 20], 4, 2, N, P, dtype, 25)
    want_y, want_s = forward(x)
    for at in (0, 15, 16, 47, 62, 130, 255, 299):
        t, rest = 40 + at, slice(40 + at, 340)
        # one channel of a head from the token on; a group's heads from it on, by a row of their
        # states; a group's heads at the token alone; a head from it on
        cases = [("x", (t, 1, 5), (rest, 1, 5), (1, 1, slice(None), 5)), ("B", (t, 1, 7), (rest, slice(2, 4)), (1, slice(2, 4), 7)),
                 ("C", (t, 0, 3), (t, slice(0, 2)), None)]
        if value != value:
            cases.append(("raw_dt", (t, 2), (rest, 2), (1, 2)))
        for name, index, rows, states in cases:
            bad = dict(x, **{name: x[name].clone()})
            bad[name][index] = value
            y, s = forward(bad)
            hit, hit_s = torch.zeros_like(y, dtype=torch.bool), torch.zeros_like(s, dtype=torch.bool)
            hit[rows] = True
            if states is not None:
                hit_s[states] = True
            assert torch.equal(y[~hit], want_y[~hit]) and torch.equal(s[~hit_s], want_s[~hit_s]), (name, at)
            assert not bool(torch.isfinite(y[hit]).any()) and not bool(torch.isfinite(s[hit_s]).any()), (name, at)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,H", [([40, 300], 2), ([2000], 1)])  # the last in segments
def test_an_infinity_stays_one_in_the_states(dtype, lens, H):
    announce("infinities in states %s %s" % (dtype, lens))
    x = make(lens, H, 1, 64, 64, dtype, 26)
    x["A_log"].fill_(-9.0)  # nothing decays away
    for at, value in ((150, float("inf")), (170, float("-inf"))):
        x["x"][at, 0, at % 64] = value
    pool = x["init"].clone()
    y = ssm_recurrent(*[x[k] for k in NAMES], pool, x["cu"])
    got, final = forward(x)
    there = torch.isinf(pool)
    assert int(there.sum()) == 128 and torch.equal(final[there], pool[there])
    assert bool(torch.isfinite(final[~there]).all())
    assert torch.equal(torch.isfinite(got), torch.isfinite(y))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_decays_past_fp32(dtype):
    announce("scan with exp(A_log) past fp32's and fp64's largest %s" % dtype)
    x = make([150, 3, 128, 64], 4, 1, 64, 64, dtype, 28)
    x["A_log"].copy_(torch.tensor([89.0, 100.0, 700.0, 1.0]))
    x["raw_dt"][5] = x["raw_dt"][149] = -float("inf")  # steps of zero
    parity(x)
    x["A_log"][0] = 1000.0
    x["raw_dt"][5] = x["raw_dt"][149] = 0.0  # the reference's exp(1000) times zero is NaN
    y_ref, s_ref = ssm_ref.scan(*[to_np(x[k]) for k in NAMES], x["cu_host"], to_np(x["init"]))
    y_abs, s_abs = reference(dict(x, A_log=x["A_log"].clamp(max=700.0)), absolute=True)[:2]
    y, final = forward(x)
    one = 1e-5 if dtype is F32 else 2.0 ** -8 + 1e-5
    held("y", y, y_ref, HALF_STEP[dtype] * np.abs(y_ref) + one * y_abs)
    held("final", final, s_ref, 1e-5 * s_abs)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 37, 63, 64, 127, 128])
def test_no_sequences_over_few_tokens(dtype, T):
    announce("scan of %d tokens in no sequence %s" % (T, dtype))
    x = make([T], 6, 1, 64, 64, dtype, 29)
    x.update(cu=torch.zeros(1, dtype=torch.int32, device="cuda"), init=None, dfinal=None)
    leave_nan(x["x"].shape, dtype)
    y, final = forward(x)
    got = backward(x)
    assert final.shape == (0, 6, 64, 64)
    for t in (y, *got[:7]):
        assert bool((t == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_gradients_of_what_is_not_a_number(dtype, value):
    announce("gradients with %s in a chunk %s" % (value, dtype))
    x = make([40, 700, 20], 4, 2, 64, 128, dtype, 27)
    want = backward(x)
    t, Q = 40 + 300, 128 if dtype is BF16 else 64
    before, behind = 40 + 300 // Q * Q, 40 + (300 // Q + 1) * Q  # its chunk
    for name, index, kept in (("x", (t, 1, 5), "before"), ("B", (t, 1, 7), "before"), ("C", (t, 1, 7), "behind"),
                              ("dy", (t, 1, 5), "behind")):
        bad = dict(x, **{name: x[name].clone()})
        bad[name][index] = value
        got = backward(bad)
        for i in (0, 1, 3, 4):  # chunks that the formulas keep free of it, and the other sequences
            a, b = (0, before) if kept == "before" else (behind, 760)
            assert torch.equal(got[i][a:b], want[i][a:b]), (name, i)
            assert torch.equal(got[i][:40], want[i][:40]) and torch.equal(got[i][740:], want[i][740:]), (name, i)
        if name == "x":  # dx and the gradients of states do not depend on x
            assert torch.equal(got[0], want[0]) and torch.equal(got[7], want[7])
        if name == "dy":  # one column of a head's states
            assert not bool(torch.isfinite(got[7][1, 1, :, 5]).any())
            got[7][1, 1, :, 5] = want[7][1, 1, :, 5]
            assert torch.equal(got[7], want[7])
        for i in (0, 1):  # the other heads: of the group in x and dy, of the other one in B and C
            others = [0, 2, 3] if name in ("x", "dy") else [0, 1]
            assert torch.equal(got[i][:, others], want[i][:, others]), (name, i)
        assert not bool(torch.isfinite(got[2]).all())
