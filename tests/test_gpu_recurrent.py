"""GPU parity of the recurrent form (kda_recurrent, gdn2_recurrent) against the
FP64 reference (needs an MI355X).

Tolerances. O is fp32 arithmetic rounded once to the dtype: each element is
within half a step of it (2^-8 of its value for bf16) plus the fp32 error,
for which 1e-5 of the row's norm is allowed, as for the chunked operator's
fp32 results: a token multiplies the state by coefficients that carry at
most about 16 roundings of 2^-24 (norm sums of 128 terms in a tree, exp,
sigmoid), 1e-6 in all, and the gate's decay keeps earlier tokens' errors
from adding up beyond a few tokens' worth. States are fp32 for either dtype:
1e-5 normalised L2.
"""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import layer_ref
from recompute_kda_chunked_amd import KdaError, gdn2_recurrent, kda_forward, kda_recurrent
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def check_rows(got, ref, dtype, what="o"):
    got, ref = to_np(got), np.asarray(ref)
    norm = np.linalg.norm(ref, axis=-1, keepdims=True) / np.sqrt(ref.shape[-1])
    off = np.abs(got - ref) - HALF_STEP[dtype] * np.abs(ref) * (1 + 1e-5) - 1e-5 * norm
    print("%s worst excess %.2e, L2 %.2e" % (what, off.max() if off.size else 0, rel(got, ref)), flush=True)
    assert np.all(off <= 0), what


def problem(lens, H, D, dtype, seed, per_head=False, gdn2=False, slots=None):
    """Inputs, a pool of states and (when `slots` is larger than the number of
    sequences) scattered slot indices."""
    x = kda_inputs.make_inputs(lens, H, D, D, dtype, seed, "cuda", A_log=0.2, dt_bias=-1.0,
                               gate_per_head=per_head, gdn2=gdn2, with_dO=False)
    n = slots or len(lens)
    x["state"] = kda_inputs.make_states(n, H, D, D, seed, "cuda")["h0"]
    gen = torch.Generator().manual_seed(seed)
    x["idx"] = None if slots is None else torch.randperm(n, generator=gen)[:len(lens)].to(torch.int32).cuda()
    return x


def run(x, cu=True, **kw):
    f, gates = (gdn2_recurrent, ("raw_b", "raw_w")) if "raw_b" in x else (kda_recurrent, ("raw_beta",))
    return f(x["q"], x["k"], x["v"], x["raw_g"], *[x[g] for g in gates], x["A_log"], x["dt_bias"],
             x["state"], x["cu_seqlens"] if cu else None, state_indices=x["idx"], **kw)


def reference(x, **kw):
    gates = {g: x[g] for g in (("raw_b", "raw_w") if "raw_b" in x else ("raw_beta",))}
    return layer_ref.recurrent(x["q"], x["k"], x["v"], x["raw_g"], x["A_log"], x["dt_bias"],
                               x["state"], x["cu_seqlens_host"], x["idx"], **gates, **kw)


def compare(x, **kw):
    o_ref, s_ref = reference(x, **kw)  # before the call: it updates the pool
    o = run(x, **kw)
    torch.cuda.synchronize()
    check_rows(o, o_ref, x["q"].dtype)
    e = rel(to_np(x["state"]), s_ref)
    print("state %.2e" % e, flush=True)
    assert e <= 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,H,slots", [([1], 1, None), ([1] * 5, 3, 9), ([3, 0, 1, 8, 0], 2, 7),
                                          ([0, 0], 1, None), ([67], 1, 3)])
def test_kda(dtype, D, lens, H, slots):
    announce("recurrent %s D%d %s H%d" % (dtype, D, lens, H))
    if sum(lens) == 0:
        x = problem([1] * len(lens), H, D, dtype, 5, slots=slots)
        x["cu_seqlens"].zero_()
        before = x["state"].clone()
        out = torch.full_like(x["v"], 7.0)
        run(x, out=out)
        assert torch.equal(before, x["state"]) and bool((out == 7).all())
        return
    compare(problem(lens, H, D, dtype, 1, slots=slots))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("mode", [0, 1])
def test_gates(dtype, per_head, mode):
    announce("recurrent gates %s per_head %s mode %d" % (dtype, per_head, mode))
    for D in (64, 128):
        compare(problem([2, 1, 5], 3, D, dtype, 2, per_head=per_head), gate_mode=mode, scale=0.3,
                lower_bound=-2.0, eps=1e-3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_gdn2(dtype, D):
    announce("recurrent gdn2 %s D%d" % (dtype, D))
    for lens in ([1, 1, 1], [4, 0, 9]):
        compare(problem(lens, 2, D, dtype, 3, gdn2=True, slots=6))


def test_one_token_each_without_cu_seqlens():
    announce("no cu_seqlens")
    x = problem([1] * 6, 2, 128, torch.bfloat16, 4, slots=8)
    y = dict(x, state=x["state"].clone())
    o_ref, s_ref = reference(x)
    # the two launches may add a column's 128 products in different orders, so
    # each is held to the reference, not to the other bit by bit
    for z, cu in ((x, False), (y, True)):
        check_rows(run(z, cu=cu), o_ref, torch.bfloat16)
        assert rel(to_np(z["state"]), s_ref) <= 1e-5


def test_padded_sequences_and_rows_behind_the_last():
    announce("padding")
    for D in (64, 128):
        x = problem([2, 1, 1, 3, 2], 2, D, torch.bfloat16, 6, slots=5)
        x["idx"][1], x["idx"][3], x["idx"][4] = -1, -7, 2147483647
        cu = [0, 2, 3, 4, 7, 7]  # the last two rows belong to no sequence
        x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        x["cu_seqlens_host"] = cu
        x["state"][int(x["idx"][0])] *= 0.5
        o_ref, s_ref = reference(x)
        out = torch.full_like(x["v"], 9.0)
        run(x, out=out)
        assert bool((out[7:] == 9).all()) and bool((out[2] == 0).all()) and bool((out[4:7] == 0).all())
        check_rows(out[:7], o_ref[:7], torch.bfloat16)
        assert rel(to_np(x["state"]), s_ref) <= 1e-5
        used = {int(i) for i in x["idx"][[0, 2]]}
        y = problem([2, 1, 1, 3, 2], 2, D, torch.bfloat16, 6, slots=5)
        for s in set(range(5)) - used:
            assert torch.equal(x["state"][s], y["state"][s])


@pytest.mark.parametrize("dtype,D,n,H", [(torch.bfloat16, 128, 130, 32), (torch.float32, 64, 65, 64)])
def test_large_decoding_batches(dtype, D, n, H):
    announce("%d sequences x %d heads D%d" % (n, H, D))  # enough blocks for the launch of large batches
    x = problem([1] * n, H, D, dtype, 17, slots=n + 5)
    some = [0, 1, n // 2, n - 1]
    part = {k: x[k][some].clone() for k in ("q", "k", "v", "raw_g", "raw_beta")}
    part.update(A_log=x["A_log"], dt_bias=x["dt_bias"], state=x["state"].clone(), idx=x["idx"][some],
                cu_seqlens_host=[0, 1, 2, 3, 4])
    o_ref, s_ref = reference(part)
    o = run(x, cu=False)
    check_rows(o[some], o_ref, dtype)
    at = x["idx"][some].long()
    assert rel(to_np(x["state"][at]), s_ref[at.cpu().numpy()]) <= 1e-5
    rest = sorted(set(range(n + 5)) - set(x["idx"].tolist()))
    assert torch.equal(x["state"][rest], part["state"][rest])


@pytest.mark.parametrize("n", [3, 70, 200])
def test_bad_slots_give_nan_and_touch_nothing(n):
    announce("slots past the pool and slots named twice, %d sequences" % n)
    lens = [1] * n
    lens[0] = 0  # a sequence without tokens takes no slot
    x = problem(lens, 2, 64, torch.bfloat16, 15, slots=n + 2)
    x["idx"][0] = x["idx"][1]
    bad = {n - 1: n + 2}
    if n > 3:
        bad.update({n - 2: int(x["idx"][1]), n // 2: int(x["idx"][2])})
    y = dict(x, state=x["state"].clone(), idx=x["idx"].clone())
    for i, s in bad.items():
        x["idx"][i], y["idx"][i] = s, -1
    got, want = run(x), run(y)
    for i in range(1, n):
        row = got[i - 1]
        assert bool(torch.isnan(row).all()) if i in bad else torch.equal(row, want[i - 1])
    assert torch.equal(x["state"], y["state"])


def test_padding_hides_nan_inputs():
    announce("nan in padded rows")
    x = problem([1, 1, 1], 2, 64, torch.float32, 7)
    x["idx"] = torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda")
    for n in ("q", "k", "v", "raw_g", "raw_beta"):
        x[n][1] = float("nan")
    before = x["state"].clone()
    o = run(x)
    assert bool((o[1] == 0).all()) and bool(torch.isfinite(o).all())
    assert torch.equal(x["state"][1], before[1])


def test_cu_seqlens_outside_the_tokens_are_clamped():
    announce("clamped cu_seqlens")
    x = problem([2, 2], 1, 64, torch.float32, 8)
    y = dict(x, state=x["state"].clone())
    x["cu_seqlens"] = torch.tensor([-5, 2, 1000], dtype=torch.int32, device="cuda")
    assert torch.equal(run(x), run(y)) and torch.equal(x["state"], y["state"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slices_of_a_fused_projection(dtype):
    announce("strided rows %s" % dtype)
    lens, H, D = [3, 1, 2], 2, 64
    for per_head, gdn2 in ((False, False), (True, False), (False, True)):
        x = problem(lens, H, D, dtype, 9, per_head=per_head, gdn2=gdn2)
        y = dict(x, state=x["state"].clone())
        names = [n for n in ("q", "k", "v", "raw_g", "raw_beta", "raw_b", "raw_w") if n in x]
        if gdn2:
            names.remove("raw_beta")
        wide = torch.full((6, sum(-(-x[n][0].numel() // 8) * 8 for n in names) + 8), float("nan"),
                          dtype=dtype, device="cuda")
        at = 8
        for n in names:
            m = x[n][0].numel()
            wide[:, at:at + m] = x[n].reshape(6, m)
            y[n] = wide[:, at:at + m].view(x[n].shape)
            at += -(-m // 8) * 8
        assert not y["q"].is_contiguous()
        assert torch.equal(run(x), run(y)) and torch.equal(x["state"], y["state"])


def test_decoding_continues_the_chunked_form():
    announce("prefill, then decode")
    for per_head in (False, True):
        H, D, lens = 2, 128, [70, 33]
        x = kda_inputs.make_inputs([n + 4 for n in lens], H, D, D, torch.float32, 10, "cuda",
                                   dt_bias=-2.0, gate_per_head=per_head)
        names = ("q", "k", "v", "raw_g", "raw_beta")
        cu = x["cu_seqlens_host"]
        whole, ht, _ = kda_forward(*[x[n] for n in names], x["A_log"], x["dt_bias"], x["cu_seqlens"],
                                   cu_seqlens_host=cu, chunk=32, output_final_state=True)
        first = torch.cat([torch.arange(a, a + n) for a, n in zip(cu, lens)]).cuda()
        pcu = [0, lens[0], sum(lens)]
        _, state, _ = kda_forward(*[x[n][first] for n in names], x["A_log"], x["dt_bias"],
                                  torch.tensor(pcu, dtype=torch.int32, device="cuda"),
                                  cu_seqlens_host=pcu, chunk=32, output_final_state=True)
        for j in range(4):
            rows = torch.tensor([a + n + j for a, n in zip(cu, lens)], device="cuda")
            o = kda_recurrent(*[x[n][rows] for n in names], x["A_log"], x["dt_bias"], state)
            assert rel(to_np(o), to_np(whole[rows])) <= 1e-5
        assert rel(to_np(state), to_np(ht)) <= 1e-5


def test_pool_and_rows_past_32_bits():
    announce("offsets past 2^31 elements")
    H, D, slots = 64, 128, 2100  # 2.2e9 state elements
    x = problem([1, 1], H, D, torch.bfloat16, 11)
    pool = torch.empty((slots, H, D, D), dtype=torch.float32, device="cuda")
    pool[0], pool[slots - 1] = x["state"][0], x["state"][1]
    small = dict(x, state=x["state"].clone())
    x["state"], x["idx"] = pool, torch.tensor([0, slots - 1], dtype=torch.int32, device="cuda")
    base = torch.empty((1 << 31) + (1 << 16), dtype=torch.bfloat16, device="cuda")
    far = base.as_strided((2, H, D), (1 << 31, D, 1))  # the second token 2^31 elements on
    far.copy_(x["q"])
    x["q"] = far
    assert torch.equal(run(x), run(small))
    assert torch.equal(pool[0], small["state"][0]) and torch.equal(pool[-1], small["state"][1])


def test_two_streams_and_graph_replay():
    announce("streams, capture and replay")
    xs = [problem([1, 2, 1], 4, 128, torch.bfloat16, s, slots=6) for s in (12, 13)]
    want = []
    for x in xs:
        y = dict(x, state=x["state"].clone())
        want.append((run(y), y["state"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    start = [x["state"].clone() for x in xs]
    torch.cuda.synchronize()
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append(run(x))
    torch.cuda.synchronize()
    for x, o, (wo, ws) in zip(xs, got, want):
        assert torch.equal(o, wo) and torch.equal(x["state"], ws)
    # the same call captured: replays advance the state, and follow the slots
    # and lengths that lie in its buffers at the time
    x = xs[0]
    x["state"].copy_(start[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(x)
    x["state"].copy_(start[0])
    y = dict(x, state=start[0].clone(), idx=x["idx"].clone(), cu_seqlens=x["cu_seqlens"].clone())
    for step in range(4):
        if step == 2:
            x["idx"].copy_(x["idx"].flip(0))
            x["cu_seqlens"].copy_(torch.tensor([0, 0, 3, 4], dtype=torch.int32))
            y["idx"], y["cu_seqlens"] = x["idx"].clone(), x["cu_seqlens"].clone()
        g.replay()
        ref = run(y)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(x["state"], y["state"])


def test_no_tokens():
    announce("no tokens")
    x = problem([1], 2, 64, torch.float32, 14)
    for n in ("q", "k", "v", "raw_g", "raw_beta"):
        x[n] = x[n][:0]
    before = x["state"].clone()
    assert run(x, cu=False).shape == (0, 2, 64)
    x["cu_seqlens"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert run(x).shape == (0, 2, 64)
    assert torch.equal(before, x["state"])


def test_state_between_its_neighbours():
    announce("a state with its inputs and its output right before and behind it")
    x = problem([2, 1, 3], 2, 64, torch.float32, 18)
    y = dict(x, state=x["state"].clone())
    names = ["q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias"]
    sizes = {n: x[n].numel() for n in names + ["state"]}
    order = ["q", "k", "v", "state", "raw_g", "raw_beta", "dt_bias", "A_log"]
    buf = torch.full((sum(sizes.values()) + x["v"].numel(),), float("nan"), device="cuda")
    at = 0
    for n in order:
        y[n] = buf[at:at + sizes[n]].view(x[n].shape)
        y[n].copy_(x[n])
        at += sizes[n]
    assert y["state"].data_ptr() == y["v"].data_ptr() + 4 * sizes["v"]
    assert torch.equal(run(y), run(x)) and torch.equal(x["state"], y["state"])
    for n in ("q", "raw_g"):  # over either end
        z = dict(y)
        i = y["state"].data_ptr() - buf.data_ptr()
        i = (i // 4 - sizes[n] + 4) if n == "q" else (i // 4 + sizes["state"] - 4)
        z[n] = buf[i:i + sizes[n]].view(x[n].shape)
        with pytest.raises(KdaError, match="kda_recurrent failed"):
            run(z)


def test_sequences_that_clamping_leaves_empty_take_no_slot():
    announce("a sequence before the first token names the slot of the next")
    x = problem([3], 2, 64, torch.float32, 19, slots=3)
    x["idx"] = x["idx"].repeat(2)
    y = dict(x, state=x["state"].clone(), idx=x["idx"][:1])
    x["cu_seqlens"] = torch.tensor([-4, -2, 3], dtype=torch.int32, device="cuda")
    assert torch.equal(run(x), run(y)) and torch.equal(x["state"], y["state"])


@pytest.mark.parametrize("n", [1026, 1200, 5000])
@pytest.mark.parametrize("cu", [False, True])
def test_bad_slots_among_many_sequences(n, cu):
    announce("slots named twice among %d sequences" % n)
    x = problem([1] * n, 1, 64, torch.float32, 21, slots=n + 2)
    first = {1023: 0, 1024: 1022, 1025: 7, n // 2 + 300: n // 2, n - 2: 1, n - 1: n - 3}  # sequence: the earlier one
    y = dict(x, state=x["state"].clone(), idx=x["idx"].clone())
    for i, j in first.items():
        x["idx"][i], y["idx"][i] = x["idx"][j], -1
    got, want = run(x, cu=cu), run(y, cu=cu)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[list(first)] = True
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[~bad])
    assert torch.equal(x["state"], y["state"])


def leave_nan(shape, dtype):
    """NaN in the memory that the next tensor of this size is given."""
    for _ in range(3):
        torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2), (128, 40)])  # the last: the wide launch
@pytest.mark.parametrize("gdn2", [False, True])
def test_new_rows_of_no_sequence_are_zero(dtype, D, H, gdn2):
    announce("rows of no sequence in a new O, %s D%d H%d gdn2 %s" % (dtype, D, H, gdn2))
    for cu in ([0, 2, 3, 3, 5], [1, 2, 2, 4, 4], [0, 0, 0, 0, 0], [23, 23, 23, 23, 23], [9, 9, 12, 12, 12]):
        x = problem([5, 6, 7, 5], H, D, dtype, 22, gdn2=gdn2, slots=6)
        x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        y = dict(x, state=x["state"].clone())
        leave_nan(x["v"].shape, dtype)
        got = run(x)
        kept = torch.full_like(x["v"], 7.0)
        run(y, out=kept)
        assert bool((kept[:cu[0]] == 7).all()) and bool((kept[cu[-1]:] == 7).all())
        assert bool((got[:cu[0]] == 0).all()) and bool((got[cu[-1]:] == 0).all())
        assert torch.equal(got[cu[0]:cu[-1]], kept[cu[0]:cu[-1]]) and torch.equal(x["state"], y["state"])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    leave_nan(x["v"].shape, dtype)
    assert bool((run(dict(x, cu_seqlens=none, idx=None)) == 0).all())


def test_replay_with_fewer_tokens_leaves_no_old_rows():
    announce("a captured call replayed with shorter sequences")
    x = problem([3, 4, 2], 2, 128, torch.bfloat16, 23, slots=5)
    y = dict(x, state=x["state"].clone())
    start = x["state"].clone()
    run(dict(x, state=start.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x)
    x["state"].copy_(start)
    for cu in ([0, 3, 7, 9], [0, 1, 3, 4], [0, 0, 0, 1], [2, 4, 4, 5], [0, 3, 7, 9]):
        x["cu_seqlens"].copy_(torch.tensor(cu, dtype=torch.int32))
        want = run(y)  # the same lengths: y holds the same cu_seqlens
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(x["state"], y["state"])
        assert bool((out[:cu[0]] == 0).all()) and bool((out[cu[-1]:] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["channel", "head", "gdn2"])
@pytest.mark.parametrize("D,H", [(128, 32), (64, 33)])
def test_ragged_tokens_of_many_heads(dtype, kind, D, H):
    announce("ragged tokens, %s %s D%d H%d" % (dtype, kind, D, H))  # more than 128 (sequence, head) pairs
    compare(problem([4, 1, 0, 8, 2], H, D, dtype, 24, per_head=kind == "head", gdn2=kind == "gdn2", slots=7))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_gdn2_without_cu_seqlens(dtype, D):
    announce("GDN-2, one token each, %s D%d" % (dtype, D))
    x = problem([1] * 5, 3, D, dtype, 25, gdn2=True, slots=9)
    o_ref, s_ref = reference(x)
    check_rows(run(x, cu=False), o_ref, dtype)
    assert rel(to_np(x["state"]), s_ref) <= 1e-5


@pytest.mark.parametrize("dtype,D,n,H,kind", [(torch.bfloat16, 128, 130, 32, "gdn2"), (torch.float32, 128, 130, 32, "gdn2"),
                                              (torch.float32, 64, 65, 64, "gdn2"), (torch.bfloat16, 64, 65, 64, "gdn2"),
                                              (torch.float32, 128, 129, 32, "channel"),
                                              (torch.bfloat16, 128, 130, 32, "head")])
def test_large_decoding_batches_of_every_form(dtype, D, n, H, kind):
    announce("%d sequences x %d heads D%d %s %s" % (n, H, D, kind, dtype))
    x = problem([1] * n, H, D, dtype, 26, per_head=kind == "head", gdn2=kind == "gdn2", slots=n + 3)
    gates = ("raw_b", "raw_w") if kind == "gdn2" else ("raw_beta",)
    some = [0, 2, n // 2, n - 1]
    part = {k: x[k][some].clone() for k in ("q", "k", "v", "raw_g", *gates)}
    part.update(A_log=x["A_log"], dt_bias=x["dt_bias"], state=x["state"].clone(), idx=x["idx"][some],
                cu_seqlens_host=[0, 1, 2, 3, 4])
    o_ref, s_ref = reference(part)
    o = run(x, cu=False)
    check_rows(o[some], o_ref, dtype)
    at = x["idx"][some].long()
    assert rel(to_np(x["state"][at]), s_ref[at.cpu().numpy()]) <= 1e-5
    rest = sorted(set(range(n + 3)) - set(x["idx"].tolist()))
    assert torch.equal(x["state"][rest], part["state"][rest])
