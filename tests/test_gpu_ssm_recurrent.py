"""GPU parity of the selective scan's decoding form (ssm_recurrent) against the
FP64 reference (needs an MI355X).

Tolerances as for the recurrent form of the delta rule: y is fp32 arithmetic
rounded once, each element within half a step of the dtype plus 1e-5 of the
row's norm (the decay and the step size carry about 10 roundings of 2^-24, the
128 products of a column are added in a tree, and decays below 1 keep earlier
tokens' errors from adding up beyond a few tokens' worth); states, fp32 for
either dtype, 1e-5 normalised L2.
"""
import pytest
import torch

from oracle import ssm_ref
from recompute_kda_chunked_amd import KdaError, ssm_recurrent
from test_gpu_recurrent import check_rows, leave_nan
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def ssm_inputs(lens, H, G, N, P, dtype, seed, slots=None, fused=False, pool=True):
    """Inputs on the GPU; with `fused` x, B and C are slices of wider rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, n = sum(lens), len(lens)

    def randn(*shape, dt=dtype):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    x, B, C = randn(T, H, P), randn(T, G, N), randn(T, G, N)
    if fused:
        wide = torch.full((T, H * P + 2 * G * N + 24), float("nan"), dtype=dtype, device="cuda")
        at, cut = 8, []
        for t in (x, B, C):
            m = t.shape[1] * t.shape[2]
            wide[:, at:at + m] = t.reshape(T, m)
            cut.append(wide[:, at:at + m].view(t.shape))
            at += m + 8
        x, B, C = cut
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    d = dict(x=x, raw_dt=randn(T, H), A_log=torch.rand(H, generator=gen, device="cuda") * 2.5, B=B, C=C,
             D=randn(H, dt=F32), dt_bias=randn(H, dt=F32) - 2.5, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             cu_host=cu, limit=(0.0, INF))
    if pool:
        d["state"] = randn(slots or n, H, N, P, dt=F32)
        d["idx"] = None if slots is None else torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32).cuda()
    return d


def run(x, cu=True, **kw):
    return ssm_recurrent(*[x[k] for k in ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias", "state")],
                         x["cu"] if cu else None, state_indices=x["idx"], dt_limit=x["limit"], **kw)


def reference(x):
    return ssm_ref.scan(*[x[k] for k in ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias")], x["cu_host"],
                        x["state"], x["idx"], x["limit"])


def compare(x, cu=True):
    y_ref, s_ref = reference(x)  # before the call: it updates the pool
    y = run(x, cu)
    check_rows(y, y_ref, x["x"].dtype, "y")
    assert rel(to_np(x["state"]), s_ref) <= 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens,H,G,slots", [([1], 1, 1, None), ([1] * 5, 6, 2, 9), ([3, 0, 1, 8, 0], 4, 1, 7),
                                            ([67], 3, 3, 3)])
def test_ssm_recurrent(dtype, N, P, lens, H, G, slots):
    announce("ssm recurrent %s N%d P%d %s H%d G%d" % (dtype, N, P, lens, H, G))
    compare(ssm_inputs(lens, H, G, N, P, dtype, 1, slots))
    if max(lens) == 1:
        compare(ssm_inputs(lens, H, G, N, P, dtype, 2, slots), cu=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_limits_and_missing_parameters(dtype):
    announce("step limits, no D, no bias %s" % dtype)
    x = ssm_inputs([2, 5], 4, 2, 64, 64, dtype, 3)
    x["limit"] = (0.05, 0.11)
    compare(x)
    for name in ("D", "dt_bias"):
        compare(dict(ssm_inputs([2, 5], 4, 2, 64, 64, dtype, 4), **{name: None}))
    x = ssm_inputs([2, 5], 4, 2, 64, 64, dtype, 5)  # steps of 1e-30 and of 90
    x["raw_dt"][:, 0], x["raw_dt"][:, 1], x["dt_bias"][:2] = -70.0, 90.0, 0.0
    compare(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_a_fused_projection(dtype):
    announce("strided rows %s" % dtype)
    x, y = (ssm_inputs([3, 1, 2], 4, 2, 128, 64, dtype, 6, slots=5, fused=f) for f in (False, True))
    assert not y["x"].is_contiguous()
    wide = torch.full((6, 12), float("nan"), dtype=dtype, device="cuda")
    wide[:, 3:7] = y["raw_dt"]
    y["raw_dt"] = wide[:, 3:7]
    assert torch.equal(run(x), run(y)) and torch.equal(x["state"], y["state"])


def test_padded_sequences_bad_slots_and_rows_of_no_sequence():
    announce("padding, bad slots, rows of no sequence")
    x = ssm_inputs([1, 2, 1, 1, 3, 2], 2, 1, 64, 64, BF16, 7, slots=8)
    x["idx"][1], x["idx"][3], x["idx"][4] = -1, 8, x["idx"][0]
    cu = [1, 2, 3, 4, 5, 7, 8]  # row 0 and the last two belong to no sequence
    x["cu"], x["cu_host"] = torch.tensor(cu, dtype=torch.int32, device="cuda"), cu
    x["x"][2], x["raw_dt"][2] = float("nan"), float("nan")  # of the padded sequence
    start = x["state"].clone()
    want = dict(x, state=start.clone(), idx=x["idx"].clone())
    want["idx"][3], want["idx"][4] = -1, -1
    y_ref, s_ref = reference(want)
    leave_nan(x["x"].shape, BF16)
    y = run(x)
    assert bool(torch.isnan(y[4:7]).all())
    y[4:7] = 0
    check_rows(y, y_ref, BF16, "y")
    assert bool((y[0] == 0).all()) and bool((y[2] == 0).all()) and bool((y[8:] == 0).all())
    assert rel(to_np(x["state"]), s_ref) <= 1e-5
    for s in set(range(8)) - {int(x["idx"][i]) for i in (0, 2, 5)}:
        assert torch.equal(x["state"][s], start[s])
    out = torch.full_like(y, 7.0)
    run(dict(x, state=start.clone()), out=out)
    assert bool((out[0] == 7).all()) and bool((out[8:] == 7).all())
    x["cu"] = torch.tensor([-5, 2, 3, 4, 5, 7, 1000], dtype=torch.int32, device="cuda")  # clamped
    z = dict(x, cu=torch.tensor([0, 2, 3, 4, 5, 7, 10], dtype=torch.int32, device="cuda"), state=x["state"].clone())
    assert torch.equal(run(x).nan_to_num(5.0), run(z).nan_to_num(5.0)) and torch.equal(x["state"], z["state"])


@pytest.mark.parametrize("cu", [False, True])
def test_many_indexed_sequences(cu):
    announce("slots named twice among 1200 sequences")
    n = 1200
    x = ssm_inputs([1] * n, 1, 1, 64, 64, F32, 8, slots=n + 2)
    y = dict(x, state=x["state"].clone(), idx=x["idx"].clone())
    for i, j in ((1100, 3), (1199, 1198)):
        x["idx"][i], y["idx"][i] = x["idx"][j], -1
    got, want = run(x, cu), run(y, cu)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[1100, 1199]] = True
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[~bad])
    assert torch.equal(x["state"], y["state"])


def test_large_batch():
    announce("130 sequences x 32 heads")
    x = ssm_inputs([1] * 130, 32, 4, 128, 64, BF16, 9, slots=133)
    some = [0, 1, 65, 129]
    part = {k: x[k][some].clone() for k in ("x", "raw_dt", "B", "C")}
    part = dict(x, **part, state=x["state"].clone(), idx=x["idx"][some], cu_host=[0, 1, 2, 3, 4])
    y_ref, s_ref = reference(part)
    y = run(x, cu=False)
    check_rows(y[some], y_ref, BF16, "y")
    at = x["idx"][some].long()
    assert rel(to_np(x["state"][at]), s_ref[at.cpu().numpy()]) <= 1e-5
    rest = sorted(set(range(133)) - set(x["idx"].tolist()))
    assert torch.equal(x["state"][rest], part["state"][rest])


def test_pool_and_rows_past_32_bits():
    announce("offsets past 2^31 elements")
    H, N, P, slots = 64, 128, 128, 2100
    x = ssm_inputs([1, 1], H, 1, N, P, BF16, 10)
    pool = torch.empty((slots, H, N, P), dtype=F32, device="cuda")
    pool[0], pool[slots - 1] = x["state"][0], x["state"][1]
    small = dict(x, state=x["state"].clone())
    x["state"], x["idx"] = pool, torch.tensor([0, slots - 1], dtype=torch.int32, device="cuda")
    base = torch.empty((1 << 31) + (1 << 16), dtype=BF16, device="cuda")
    for name in ("x", "B"):  # the second token 2^31 elements on
        far = base.as_strided((2, *x[name].shape[1:]), (1 << 31, x[name].shape[2], 1), 0 if name == "x" else 16384)
        far.copy_(x[name])
        x[name] = far
    assert torch.equal(run(x), run(small))
    assert torch.equal(pool[0], small["state"][0]) and torch.equal(pool[-1], small["state"][1])


def test_capture_streams_and_no_tokens():
    announce("capture and replay, two streams, no tokens")
    xs = [ssm_inputs([3, 4, 2], 2, 1, 128, 64, BF16, s, slots=5) for s in (11, 12)]
    want = []
    for x in xs:
        y = dict(x, state=x["state"].clone())
        want.append((run(y), y["state"]))
    start = [x["state"].clone() for x in xs]
    torch.cuda.synchronize()
    got = []
    for x in xs:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(run(x))
    torch.cuda.synchronize()
    for x, o, (wo, ws) in zip(xs, got, want):
        assert torch.equal(o, wo) and torch.equal(x["state"], ws)
    x = xs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x)
    x["state"].copy_(start[0])
    y = dict(x, state=start[0].clone())
    for cu in ([0, 3, 7, 9], [0, 1, 3, 4], [0, 0, 0, 1], [2, 4, 4, 5]):
        x["cu"].copy_(torch.tensor(cu, dtype=torch.int32))  # y holds the same tensor
        x["idx"].copy_(x["idx"].flip(0))
        ref = run(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(x["state"], y["state"])
    none = dict(x, **{k: x[k][:0] for k in ("x", "raw_dt", "B", "C")})
    before = x["state"].clone()
    none["cu"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert run(none).shape == (0, 2, 64) and torch.equal(before, x["state"])


def test_a_pool_over_an_input_is_refused():
    announce("a pool that overlaps an input")
    x = ssm_inputs([2], 2, 1, 64, 64, F32, 13)
    x["x"] = x["state"].view(-1)[-256:].view(2, 2, 64)
    with pytest.raises(KdaError, match="kda_ssm_recurrent failed"):
        run(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decays_past_fp32(dtype):
    announce("exp(A_log) past fp32's largest, steps of zero %s" % dtype)
    x = ssm_inputs([6, 1], 4, 1, 64, 64, dtype, 14)
    x["A_log"].copy_(torch.tensor([89.0, 100.0, 700.0, 1.0]))
    x["raw_dt"][2] = x["raw_dt"][6] = -float("inf")
    compare(x)
