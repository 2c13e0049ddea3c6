"""Refusals of a state-space layer's operators, without a GPU: the C entry
points on made-up pointers (validation comes before any launch), the binding's
checks, and what autograd and its neighbours make of a call whose launch is
left out."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from recompute_kda_chunked_amd import KdaError, _lib, group_norm, ssm, ssm_recurrent, ssm_scan, ssm_scan_backward
from test_abi import lib  # noqa: F401  (fixture)

FAKE, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
INF, NAN = float("inf"), float("nan")


def problem(**kw):
    d = dict(n_seqs=3, total_tokens=3, H=4, G=2, N=128, P=64, dtype=_lib.KDA_BF16, dt_min=0.0, dt_max=INF, n_slots=4)
    d.update(kw)
    return _lib.KdaSsmProblem(**d)


BAD = [
    (dict(n_seqs=-1), _lib.KDA_ERR_INVALID),
    (dict(total_tokens=-1), _lib.KDA_ERR_INVALID),
    (dict(H=0), _lib.KDA_ERR_INVALID),
    (dict(G=0), _lib.KDA_ERR_INVALID),
    (dict(G=3), _lib.KDA_ERR_INVALID),
    (dict(N=96), _lib.KDA_ERR_UNSUPPORTED),
    (dict(P=32), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dt_min=-0.1), _lib.KDA_ERR_INVALID),
    (dict(dt_min=0.2, dt_max=0.1), _lib.KDA_ERR_INVALID),
    (dict(dt_min=INF), _lib.KDA_ERR_INVALID),
    (dict(dt_max=NAN), _lib.KDA_ERR_INVALID),
    (dict(x_stride=255), _lib.KDA_ERR_INVALID),   # shorter than a row
    (dict(x_stride=260), _lib.KDA_ERR_INVALID),   # 520 bytes
    (dict(dt_stride=3), _lib.KDA_ERR_INVALID),
    (dict(B_stride=252), _lib.KDA_ERR_INVALID),
    (dict(C_stride=-256), _lib.KDA_ERR_INVALID),
]


def call_rec(lib, p, cu=NUL, idx=NUL, **null):  # noqa: F811
    at = lambda n: NUL if n in null else FAKE  # noqa: E731
    return lib.kda_ssm_recurrent(ctypes.byref(p) if p is not None else None,
                                 *[at(n) for n in ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias")], cu, idx,
                                 at("state"), at("y"), NUL)


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(total_tokens=4), _lib.KDA_ERR_INVALID),           # no cu_seqlens: one token each
    (dict(n_slots=2), _lib.KDA_ERR_INVALID),                # no indices: slot n of sequence n
    (dict(n_slots=-1), _lib.KDA_ERR_INVALID),
    (dict(H=1 << 23, G=1 << 23), _lib.KDA_ERR_UNSUPPORTED),  # sequences * H of 2^24 or more
])
def test_recurrent_rejects(lib, kw, code):  # noqa: F811
    assert call_rec(lib, problem(**kw)) == code


def test_recurrent_null_pointers_and_empty_calls(lib):  # noqa: F811
    assert call_rec(lib, None) == _lib.KDA_ERR_INVALID
    for n in ("x", "raw_dt", "A_log", "B", "C", "state", "y"):
        assert call_rec(lib, problem(), **{n: 1}) == _lib.KDA_ERR_INVALID
    assert call_rec(lib, problem(), D=1, dt_bias=1) == _lib.KDA_ERR_INVALID  # the state lies over x
    assert call_rec(lib, problem(n_seqs=65537, n_slots=1), cu=FAKE, idx=FAKE) == _lib.KDA_ERR_UNSUPPORTED
    # nothing to do: no launch, whatever the pointers
    assert call_rec(lib, problem(n_seqs=0, total_tokens=0)) == _lib.KDA_OK
    assert call_rec(lib, problem(total_tokens=0), cu=FAKE) == _lib.KDA_OK
    assert call_rec(lib, problem(n_seqs=0, total_tokens=5), cu=FAKE) == _lib.KDA_OK


FWD = ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias", "cu", "init", "y", "final")
BWD = FWD[:9] + ("dy", "dfinal", "dx", "draw_dt", "dA_log", "dB", "dC", "dD", "ddt_bias", "dinit")


def call_scan(lib, p, bwd, ws=1 << 44, workspace=FAKE, **null):  # noqa: F811
    fn = lib.kda_ssm_bwd if bwd else lib.kda_ssm_fwd
    return fn(ctypes.byref(p) if p is not None else None, *[NUL if n in null else FAKE for n in (BWD if bwd else FWD)],
              workspace, ws, NUL)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", BAD + [
    (dict(total_tokens=1 << 31), _lib.KDA_ERR_INVALID),
    (dict(x_stride=1 << 22), _lib.KDA_ERR_UNSUPPORTED),     # a chunk's rows in 32 bits
    (dict(B_stride=1 << 22), _lib.KDA_ERR_UNSUPPORTED),
    (dict(C_stride=(1 << 22) + 8), _lib.KDA_ERR_UNSUPPORTED),
    (dict(H=1 << 16, G=1), _lib.KDA_ERR_UNSUPPORTED),       # H * P
    (dict(H=1 << 15, G=1 << 15), _lib.KDA_ERR_UNSUPPORTED),  # G * N
    (dict(total_tokens=(1 << 31) - 1), _lib.KDA_ERR_UNSUPPORTED),
    (dict(n_seqs=1 << 21), _lib.KDA_ERR_UNSUPPORTED),       # 2^23 (chunk, head)
    (dict(P=128, n_seqs=1 << 20), _lib.KDA_ERR_UNSUPPORTED),  # 2^24 blocks of both state passes
])
def test_scan_rejects(lib, bwd, kw, code):  # noqa: F811
    p = problem(**kw)
    assert call_scan(lib, p, bwd) == code
    assert (lib.kda_ssm_bwd_workspace_bytes if bwd else lib.kda_ssm_fwd_workspace_bytes)(ctypes.byref(p)) == 0


@pytest.mark.parametrize("bwd", [False, True])
def test_scan_null_pointers_and_workspace(lib, bwd):  # noqa: F811
    size = lib.kda_ssm_bwd_workspace_bytes if bwd else lib.kda_ssm_fwd_workspace_bytes
    assert call_scan(lib, None, bwd) == _lib.KDA_ERR_INVALID and size(None) == 0
    p = problem(total_tokens=300)
    need = size(ctypes.byref(p))
    assert need > 0
    assert call_scan(lib, p, bwd, ws=need - 1) == _lib.KDA_ERR_WORKSPACE
    assert call_scan(lib, p, bwd, workspace=NUL) == _lib.KDA_ERR_INVALID
    assert call_scan(lib, p, bwd, cu=1) == _lib.KDA_ERR_INVALID  # three sequences without cu_seqlens
    for n in ("dy", "dx", "draw_dt", "dA_log", "dB", "dC") if bwd else ("y",):
        assert call_scan(lib, p, bwd, ws=need, **{n: 1}) == _lib.KDA_ERR_INVALID
    for n in ("x", "raw_dt", "A_log", "B", "C"):
        assert call_scan(lib, p, bwd, ws=need, **{n: 1}) == _lib.KDA_ERR_INVALID
    if bwd:  # the sums are written whatever there is
        assert call_scan(lib, problem(n_seqs=0, total_tokens=0), bwd, dA_log=1) == _lib.KDA_ERR_INVALID
    else:  # nothing to do: no launch, whatever the pointers
        none = {n: 1 for n in FWD if n != "cu"}
        assert call_scan(lib, problem(n_seqs=0, total_tokens=0), bwd, **none) == _lib.KDA_OK
        assert call_scan(lib, problem(total_tokens=0), bwd, **none) == _lib.KDA_OK


def test_scan_workspace_follows_the_tokens(lib):  # noqa: F811
    """Short sequences need no segments, long ones few: the room stays near the
    states' (fp32, two of them backward), a slot a chunk or sequence."""
    for dtype, Q, kept in ((_lib.KDA_BF16, 128, 2), (_lib.KDA_F32, 64, 4)):
        for n, T in ((1, 100), (1, 1 << 15), (1, 1 << 18), (8, 1 << 15), (1000, 1 << 12), (4000, 1 << 15)):
            p = problem(n_seqs=n, total_tokens=T, dtype=dtype, H=64, G=1)
            slots = T // Q + n
            states = slots * 64 * 64 * 128
            steps = slots * 64 * Q * 16
            fwd, bwd = (f(ctypes.byref(p)) for f in (lib.kda_ssm_fwd_workspace_bytes, lib.kda_ssm_bwd_workspace_bytes))
            assert states * kept <= fwd <= 2 * states * 4 + steps + (1 << 20)
            assert states * 8 <= bwd <= 3 * states * 4 + 2 * steps + 4 * slots * 64 * 5 + 256 * 64 * Q * 128 * 8 + (1 << 20)


def norm_problem(**kw):
    d = dict(rows=5, C=512, groups=8, dtype=_lib.KDA_BF16, gate=0, activation=_lib.KDA_ACT_SILU, center=1, eps=1e-6)
    d.update(kw)
    return _lib.KdaGroupNormProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _lib.KDA_ERR_INVALID),
    (dict(rows=(1 << 31) + 1), _lib.KDA_ERR_UNSUPPORTED),
    (dict(C=0), _lib.KDA_ERR_INVALID),
    (dict(groups=0), _lib.KDA_ERR_INVALID),
    (dict(groups=7), _lib.KDA_ERR_INVALID),
    (dict(C=96, groups=8), _lib.KDA_ERR_UNSUPPORTED),       # 12 channels
    (dict(C=8200, groups=1), _lib.KDA_ERR_UNSUPPORTED),
    (dict(C=1 << 21, groups=512), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate=3), _lib.KDA_ERR_UNSUPPORTED),
    (dict(activation=3), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate=1, activation=_lib.KDA_ACT_NONE), _lib.KDA_ERR_UNSUPPORTED),
    (dict(eps=-1.0), _lib.KDA_ERR_INVALID),
    (dict(eps=NAN), _lib.KDA_ERR_INVALID),
    (dict(x_stride=511), _lib.KDA_ERR_INVALID),
    (dict(gate_stride=516), _lib.KDA_ERR_INVALID),
])
def test_group_norm_rejects(lib, kw, code):  # noqa: F811
    p = ctypes.byref(norm_problem(**kw))
    gate = FAKE if kw.get("gate") else NUL
    assert lib.kda_group_norm_fwd(p, FAKE, gate, FAKE, FAKE, FAKE, NUL) == code
    assert lib.kda_group_norm_bwd(p, FAKE, gate, FAKE, FAKE, FAKE, FAKE, gate, FAKE, FAKE, FAKE, 1 << 40, NUL) == code
    assert lib.kda_group_norm_bwd_workspace_bytes(p) == 0


def test_group_norm_null_pointers_and_workspace(lib):  # noqa: F811
    for gate in (0, 1, 2):
        p, g = ctypes.byref(norm_problem(gate=gate)), FAKE if gate else NUL
        full = [FAKE, g, FAKE, NUL, FAKE]
        for i in (0, 2, 4):
            assert lib.kda_group_norm_fwd(p, *[NUL if j == i else a for j, a in enumerate(full)], NUL) == _lib.KDA_ERR_INVALID
        assert lib.kda_group_norm_fwd(p, FAKE, NUL if gate else FAKE, FAKE, NUL, FAKE, NUL) == _lib.KDA_ERR_INVALID
        need = lib.kda_group_norm_bwd_workspace_bytes(p)
        assert need > 0
        full = [FAKE, g, FAKE, NUL, FAKE, FAKE, g, FAKE, NUL, FAKE]
        assert lib.kda_group_norm_bwd(p, *full, need - 1, NUL) == _lib.KDA_ERR_WORKSPACE
        for i in (0, 2, 4, 5, 7, 9) + ((1, 6) if gate else ()):
            args = [NUL if j == i else a for j, a in enumerate(full)]
            assert lib.kda_group_norm_bwd(p, *args, need, NUL) == _lib.KDA_ERR_INVALID
    assert lib.kda_group_norm_fwd(ctypes.byref(norm_problem(rows=0)), NUL, NUL, NUL, NUL, NUL, NUL) == _lib.KDA_OK
    assert lib.kda_group_norm_bwd_workspace_bytes(None) == 0


# ------------------------------------------------------------------ the binding


def rec_inputs(T=3, H=4, G=2, N=64, P=128, dtype=torch.float32):
    z = lambda *s: torch.zeros(s, dtype=dtype)  # noqa: E731
    return dict(x=z(T, H, P), raw_dt=z(T, H), A_log=torch.zeros(H), B=z(T, G, N), C=z(T, G, N), D=torch.zeros(H),
                dt_bias=torch.zeros(H), state=torch.zeros(T, H, N, P))


def scan_inputs():
    x = rec_inputs()
    x["initial_state"] = x.pop("state")[:1].contiguous()
    return x


def norm_inputs():
    return dict(x=torch.zeros(4, 96), weight=torch.zeros(96), bias=torch.zeros(96), gate=torch.zeros(4, 96))


def norm(**x):
    return group_norm(**x, groups=3)


DIFFERENTIABLE = [(norm, norm_inputs), (ssm_scan, scan_inputs)]
IN_PLACE = [(ssm_recurrent, rec_inputs)]


@pytest.fixture
def no_launch(monkeypatch):
    calls = []
    monkeypatch.setattr(ssm, "_dev", lambda t, name: t.device)
    monkeypatch.setattr(ssm, "_call", lambda dev, name, *args, **kw: calls.append(name))
    monkeypatch.setattr(ssm, "_workspace", lambda *args: None)
    return calls


@pytest.mark.parametrize("change,match", [
    (dict(x=torch.zeros(3, 512)), "expected \\[T,H,P\\]"),
    (dict(x=torch.zeros(3, 4, 128, dtype=torch.float16)), "float32 or bfloat16"),
    (dict(raw_dt=torch.zeros(3, 2)), "raw_dt: expected"),
    (dict(raw_dt=torch.zeros(3, 4).bfloat16()), "raw_dt: expected"),
    (dict(A_log=torch.zeros(4).bfloat16()), "A_log: expected"),
    (dict(B=torch.zeros(3, 2, 128)), "C: expected"),
    (dict(C=torch.zeros(4, 2, 64)), "C: expected"),
    (dict(B=torch.zeros(3, 3, 64), C=torch.zeros(3, 3, 64)), "must divide the heads"),
    (dict(B=torch.zeros(3, 2, 32), C=torch.zeros(3, 2, 32)), "not built"),
    (dict(x=torch.zeros(3, 4, 32)), "not built"),
    (dict(D=torch.zeros(2)), "D: expected"),
    (dict(dt_bias=torch.zeros(4, 1)), "dt_bias: expected"),
    (dict(dt_limit=(0.2, 0.1)), "dt_limit"),
    (dict(dt_limit=(-0.2, 0.1)), "dt_limit"),
    (dict(dt_limit=(0.0, NAN)), "dt_limit"),
    (dict(state=torch.zeros(3, 4, 64)), "state: expected"),
    (dict(state=torch.zeros(3, 4, 128, 64)), "state: expected"),
    (dict(state=torch.zeros(2, 4, 64, 128)), "2 slots for 3 sequences"),
    (dict(state=torch.zeros(3, 4, 64, 129)[..., :128]), "state must be contiguous"),
    (dict(x=torch.zeros(3, 4, 130)[..., :128]), "elements of a token must be contiguous"),
    (dict(x=torch.zeros(1, 4, 128).expand(3, 4, 128)), "tokens overlap"),
    (dict(B=torch.zeros(3 * 128 + 1)[1:].view(3, 2, 64)), "multiples of 16 bytes"),
    (dict(C=torch.zeros(3, 129)[:, :128].view(3, 2, 64)), "multiples of 16 bytes"),
    (dict(cu_seqlens=torch.zeros(3)), "cu_seqlens: expected int32"),
    (dict(state_indices=torch.zeros(3)), "state_indices: expected"),
    (dict(out=torch.zeros(3, 4, 64)), "out: expected"),
    (dict(x=torch.zeros(3, 4, 128, requires_grad=True)), "not differentiable"),
    (dict(D=torch.zeros(4, requires_grad=True)), "not differentiable"),
])
def test_recurrent_binding_refuses(no_launch, change, match):
    with pytest.raises(KdaError, match=match):
        ssm_recurrent(**dict(rec_inputs(), **change))
    assert not no_launch


@pytest.mark.parametrize("change,match", [
    (dict(x=torch.zeros(3, 512)), "expected \\[T,H,P\\]"),
    (dict(x=torch.zeros(3, 4, 128, dtype=torch.float16)), "float32 or bfloat16"),
    (dict(raw_dt=torch.zeros(3, 4).bfloat16()), "raw_dt: expected"),
    (dict(B=torch.zeros(3, 3, 64), C=torch.zeros(3, 3, 64)), "must divide the heads"),
    (dict(C=torch.zeros(4, 2, 64)), "C: expected"),
    (dict(x=torch.zeros(3, 4, 32)), "not built"),
    (dict(dt_limit=(INF, INF)), "dt_limit"),
    (dict(initial_state=torch.zeros(3, 4, 64, 128)), "initial_state: expected"),
    (dict(initial_state=torch.zeros(1, 4, 64, 128).bfloat16()), "initial_state: expected"),
    (dict(initial_state=torch.zeros(1, 4, 128, 64).transpose(2, 3)), "contiguous"),
    (dict(cu_seqlens=torch.zeros(2)), "cu_seqlens: expected"),
    (dict(cu_seqlens=torch.zeros(0, dtype=torch.int32)), "cu_seqlens: expected"),
    (dict(cu_seqlens=torch.zeros(2, 1, dtype=torch.int32)), "cu_seqlens: expected"),
    (dict(x=torch.zeros(3, 4, 130)[..., :128]), "elements of a token must be contiguous"),
    (dict(C=torch.zeros(3, 129)[:, :128].view(3, 2, 64)), "multiples of 16 bytes"),
])
def test_scan_binding_refuses(no_launch, change, match):
    x = dict(scan_inputs(), **change)
    with pytest.raises(KdaError, match=match):
        ssm_scan(**x)
    args = [x[k] for k in ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias")]
    with pytest.raises(KdaError, match=match):
        ssm_scan_backward(*args, torch.zeros_like(x["x"]), x.get("cu_seqlens"), initial_state=x["initial_state"],
                          **{k: x[k] for k in ("dt_limit",) if k in x})
    assert not no_launch


def test_scan_gradients_must_match(no_launch):
    x = scan_inputs()
    args = [x[k] for k in ("x", "raw_dt", "A_log", "B", "C", "D", "dt_bias")]
    ssm_scan_backward(*args, torch.zeros(3, 4, 128), d_final_state=torch.zeros(1, 4, 64, 128))
    for dy, dfinal, match in ((torch.zeros(3, 512), None, "dy: expected"),
                              (torch.zeros(3, 4, 128).bfloat16(), None, "dy: expected"),
                              (torch.zeros(3, 4, 129)[..., :128], None, "dy must be contiguous"),
                              (torch.zeros(3, 4, 128), torch.zeros(2, 4, 64, 128), "d_final_state: expected")):
        with pytest.raises(KdaError, match=match):
            ssm_scan_backward(*args, dy, d_final_state=dfinal)


def test_recurrent_out_must_be_apart(no_launch):
    x = rec_inputs()
    with pytest.raises(KdaError, match="must not overlap"):
        ssm_recurrent(**x, out=x["x"])
    out = torch.zeros(3, 4, 128)
    assert ssm_recurrent(**x, out=out) is out
    x["D"] = x["dt_bias"] = None
    ssm_recurrent(**x)


@pytest.mark.parametrize("change,match", [
    (dict(x=torch.zeros(4, 96).half()), "float32 or bfloat16"),
    (dict(weight=torch.zeros(95)), "weight: expected"),
    (dict(bias=torch.zeros(96).bfloat16()), "bias: expected"),
    (dict(gate=torch.zeros(4, 48)), "gate: expected"),
    (dict(gate=None, gate_first=True), "gate_first takes a gate"),
    (dict(activation="relu"), "activation must be"),
    (dict(activation="none"), "a gate takes"),
    (dict(groups=5), "must divide"),
    (dict(groups=0), "must divide"),
    (dict(groups=8), "multiples of 8"),
    (dict(x=torch.zeros(4, 100)[:, :96], gate=None), None),
    (dict(x=torch.zeros(4, 98)[:, :96]), "multiples of 16 bytes"),
    (dict(x=torch.zeros(96, 4).t()), "must be contiguous"),
    (dict(x=torch.zeros(2, 2, 192)[..., :96], gate=None), "must be contiguous"),
])
def test_group_norm_binding_refuses(no_launch, change, match):
    x = dict(dict(norm_inputs(), groups=3), **change)
    if match is None:
        group_norm(**x)
        return
    with pytest.raises(KdaError, match=match):
        group_norm(**x)


def test_tensors_of_the_host_are_refused():
    for fn, make in IN_PLACE + DIFFERENTIABLE:
        with pytest.raises(KdaError, match="GPU device"):
            fn(**make())


@pytest.mark.parametrize("fn,make", DIFFERENTIABLE)
def test_forward_mode_and_traces_of_differentiable_calls(no_launch, fn, make):
    for name in make():
        with forward_ad.dual_level():
            x = make()
            x[name] = forward_ad.make_dual(x[name], torch.ones_like(x[name]))
            with pytest.raises(NotImplementedError, match="jvp"):
                fn(**x)
    names = list(make())
    no_launch.clear()
    traced = torch.jit.trace(lambda *t: fn(**dict(zip(names, t))), tuple(make().values()), check_trace=False)
    assert any(n.kind() == "prim::PythonOp" for n in traced.graph.nodes()) and len(no_launch) == 1
    traced(*make().values())
    assert len(no_launch) == 2


@pytest.mark.parametrize("fn,make", IN_PLACE)
def test_decoding_forms_as_autograd_sees_them(no_launch, fn, make):
    names = list(make())
    with pytest.raises(KdaError, match="cannot be traced"):
        torch.jit.trace(lambda *t: fn(**dict(zip(names, t))), tuple(make().values()), check_trace=False)
    for name in names:
        with forward_ad.dual_level():
            x = make()
            x[name] = forward_ad.make_dual(x[name], torch.ones_like(x[name]))
            with pytest.raises(KdaError, match="not differentiable"):
                fn(**x)
    for name in ("state", "out"):  # a backward that kept what a call overwrites raises
        x = make()
        if name == "out":
            x["out"] = fn(**x)
        loss = (torch.ones((), requires_grad=True) * x[name]).sum()
        versions = {n: t._version for n, t in x.items()}
        fn(**x)
        assert all(t._version == versions[n] for n, t in x.items() if n not in ("state", "out"))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
