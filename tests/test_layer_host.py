"""Refusals of the operators around the chunked one, without a GPU: the C
entry points on made-up pointers (validation comes before any launch), and
the binding's checks of shapes, types and placement."""
import ctypes

import pytest
import torch

from recompute_kda_chunked_amd import (KdaError, _lib, block_norm, gated_norm, gdn2_recurrent,
                                       kda_recurrent, short_conv, short_conv_update)
from test_abi import lib  # noqa: F401  (fixture)

FAKE, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)


# ------------------------------------------------------------------ recurrent


def rec(**kw):
    d = dict(n_seqs=3, total_tokens=3, H=2, K=128, V=128, dtype=_lib.KDA_BF16, gate_mode=0,
             scale=1.0, gate_lower_bound=-5.0, l2_eps=1e-6, n_slots=4)
    d.update(kw)
    return _lib.KdaRecurrentProblem(**d)


def call_rec(lib, p, cu=NUL, idx=NUL, g2=False, **null):  # noqa: F811
    names = ["q", "k", "v", "raw_g"] + (["raw_b", "raw_w"] if g2 else ["raw_beta"]) + ["A_log", "dt_bias"]
    args = [NUL if n in null else FAKE for n in names]
    tail = [NUL if n in null else FAKE for n in ("state", "o")]
    fn = lib.kda_gdn2_recurrent if g2 else lib.kda_recurrent
    return fn(ctypes.byref(p) if p is not None else None, *args, cu, idx, *tail, NUL)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), _lib.KDA_ERR_INVALID),
    (dict(total_tokens=-1), _lib.KDA_ERR_INVALID),
    (dict(total_tokens=4), _lib.KDA_ERR_INVALID),           # no cu_seqlens: one token each
    (dict(H=0), _lib.KDA_ERR_INVALID),
    (dict(n_slots=2), _lib.KDA_ERR_INVALID),                # no indices: slot n of sequence n
    (dict(n_slots=-1), _lib.KDA_ERR_INVALID),
    (dict(K=96, V=96), _lib.KDA_ERR_UNSUPPORTED),
    (dict(K=64), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dtype=3), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate_mode=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate_lower_bound=-6.0), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate_lower_bound=0.0), _lib.KDA_ERR_INVALID),
    (dict(gate_lower_bound=float("nan")), _lib.KDA_ERR_INVALID),
    (dict(l2_eps=-1.0), _lib.KDA_ERR_INVALID),
    (dict(scale=float("inf")), _lib.KDA_ERR_INVALID),
    (dict(q_stride=255), _lib.KDA_ERR_INVALID),             # shorter than a row
    (dict(k_stride=260), _lib.KDA_ERR_INVALID),             # 520 bytes
    (dict(v_stride=-256), _lib.KDA_ERR_INVALID),
    (dict(g_stride=257), _lib.KDA_ERR_INVALID),
    (dict(beta_stride=1), _lib.KDA_ERR_INVALID),
    (dict(H=1 << 23, n_seqs=3), _lib.KDA_ERR_UNSUPPORTED),  # N * H of 2^24 or more
])
def test_recurrent_rejects(lib, kw, code):  # noqa: F811
    assert call_rec(lib, rec(**kw)) == code


def test_recurrent_null_pointers_and_empty_calls(lib):  # noqa: F811
    assert call_rec(lib, None) == _lib.KDA_ERR_INVALID
    for n in ("q", "k", "v", "raw_g", "raw_beta", "A_log", "dt_bias", "state", "o"):
        assert call_rec(lib, rec(), **{n: 1}) == _lib.KDA_ERR_INVALID
    for n in ("raw_b", "raw_w"):
        assert call_rec(lib, rec(), g2=True, **{n: 1}) == _lib.KDA_ERR_INVALID
    assert call_rec(lib, rec(gate_mode=_lib.KDA_GATE_PER_HEAD), g2=True) == _lib.KDA_ERR_UNSUPPORTED
    assert call_rec(lib, rec(b_stride=8), g2=True) == _lib.KDA_ERR_INVALID
    # nothing to do: no launch, whatever the pointers
    assert call_rec(lib, rec(n_seqs=0, total_tokens=0)) == _lib.KDA_OK
    assert call_rec(lib, rec(total_tokens=0), cu=FAKE) == _lib.KDA_OK
    assert call_rec(lib, rec(n_seqs=0, total_tokens=5), cu=FAKE) == _lib.KDA_OK


def rec_inputs(T=3, H=2, D=64, dtype=torch.float32):
    g = lambda *s: torch.zeros(s, dtype=dtype)  # noqa: E731
    return dict(q=g(T, H, D), k=g(T, H, D), v=g(T, H, D), raw_g=g(T, H, D), raw_beta=g(T, H),
                A_log=torch.zeros(H), dt_bias=torch.zeros(H, D), state=torch.zeros(T, H, D, D))


@pytest.mark.parametrize("name,value,match", [
    ("q", torch.zeros(3, 128), "q, k"),
    ("k", torch.zeros(3, 2, 32), "k: expected"),
    ("v", torch.zeros(3, 1, 64), "v: expected"),
    ("raw_g", torch.zeros(2, 2), "raw_g: expected"),
    ("raw_beta", torch.zeros(3, 2, 1), "raw_beta: expected"),
    ("raw_beta", torch.zeros(3, 2, dtype=torch.float64), "raw_beta: expected"),
    ("A_log", torch.zeros(2, dtype=torch.bfloat16), "A_log: expected"),
    ("dt_bias", torch.zeros(2), "dt_bias: expected"),
    ("state", torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16), "state: expected"),
    ("state", torch.zeros(3, 2, 64), "state"),
    ("out", torch.zeros(3, 2, 32), "out: expected"),
    ("state", torch.zeros(3, 2, 64, 64, requires_grad=True), "not differentiable"),
    ("q", torch.zeros(3, 2, 64, requires_grad=True), "not differentiable"),
])
def test_recurrent_binding_refuses(name, value, match):
    with pytest.raises(KdaError, match=match):
        kda_recurrent(**dict(rec_inputs(), **{name: value}))


def test_recurrent_binding_refuses_host_tensors_and_other_types():
    with pytest.raises(KdaError, match="GPU"):
        kda_recurrent(**rec_inputs())
    with pytest.raises(KdaError, match="float32 or bfloat16"):
        kda_recurrent(**{n: t.half() for n, t in rec_inputs().items()})
    x = rec_inputs()
    x.pop("raw_beta")
    with pytest.raises(KdaError, match="raw_w: expected"):
        gdn2_recurrent(raw_b=x["q"], raw_w=x["q"][:2], **x)


# ------------------------------------------------------------------ norms


def gn(**kw):
    d = dict(rows=6, V=128, dtype=_lib.KDA_BF16, activation=_lib.KDA_ACT_SIGMOID, eps=1e-6)
    d.update(kw)
    return _lib.KdaGatedNormProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), _lib.KDA_ERR_INVALID),
    (dict(eps=-1.0), _lib.KDA_ERR_INVALID),
    (dict(eps=float("nan")), _lib.KDA_ERR_INVALID),
    (dict(V=0), _lib.KDA_ERR_INVALID),
    (dict(V=96), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(activation=_lib.KDA_ACT_NONE), _lib.KDA_ERR_UNSUPPORTED),
])
def test_gated_norm_rejects(lib, kw, code):  # noqa: F811
    p = ctypes.byref(gn(**kw))
    assert lib.kda_gated_norm_fwd(p, *[FAKE] * 4, NUL) == code
    assert lib.kda_gated_norm_bwd(p, *[FAKE] * 7, FAKE, 1 << 30, NUL) == code
    assert lib.kda_gated_norm_bwd_workspace_bytes(p) == 0


def test_gated_norm_null_pointers_and_workspace(lib):  # noqa: F811
    p = ctypes.byref(gn())
    need = lib.kda_gated_norm_bwd_workspace_bytes(p)
    assert need > 0
    for i in range(4):
        args = [FAKE] * 4
        args[i] = NUL
        assert lib.kda_gated_norm_fwd(p, *args, NUL) == _lib.KDA_ERR_INVALID
    for i in range(7):
        args = [FAKE] * 7
        args[i] = NUL
        assert lib.kda_gated_norm_bwd(p, *args, FAKE, need, NUL) == _lib.KDA_ERR_INVALID
    assert lib.kda_gated_norm_bwd(p, *[FAKE] * 7, FAKE, need - 1, NUL) == _lib.KDA_ERR_WORKSPACE
    assert lib.kda_gated_norm_fwd(ctypes.byref(gn(rows=0)), *[NUL] * 4, NUL) == _lib.KDA_OK


def bn(**kw):
    d = dict(tokens=5, D=256, dtype=_lib.KDA_BF16, gate=_lib.KDA_BLOCK_GATE_CHANNEL,
             residual_scale=0.5, eps=1e-6)
    d.update(kw)
    return _lib.KdaBlockNormProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), _lib.KDA_ERR_INVALID),
    (dict(eps=-1.0), _lib.KDA_ERR_INVALID),
    (dict(residual_scale=float("inf")), _lib.KDA_ERR_INVALID),
    (dict(D=0), _lib.KDA_ERR_INVALID),
    (dict(D=12), _lib.KDA_ERR_UNSUPPORTED),
    (dict(D=8200), _lib.KDA_ERR_UNSUPPORTED),
    (dict(dtype=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate=3), _lib.KDA_ERR_UNSUPPORTED),
    (dict(gate=_lib.KDA_BLOCK_GATE_NONE), _lib.KDA_ERR_INVALID),  # a gate is given
])
def test_block_norm_rejects(lib, kw, code):  # noqa: F811
    p = ctypes.byref(bn(**kw))
    assert lib.kda_block_norm_fwd(p, *[FAKE] * 7, NUL) == code
    assert lib.kda_block_norm_bwd(p, *[FAKE] * 12, FAKE, 1 << 30, NUL) == code


def test_block_norm_null_pointers_and_workspace(lib):  # noqa: F811
    p = ctypes.byref(bn())
    need = lib.kda_block_norm_bwd_workspace_bytes(p)
    for i, optional in enumerate((0, 0, 0, 1, 0, 0, 0)):  # w_post may be null
        args = [FAKE] * 7
        args[i] = NUL
        if not optional:
            assert lib.kda_block_norm_fwd(p, *args, NUL) == _lib.KDA_ERR_INVALID
    for i, optional in enumerate((0, 0, 0, 1, 0, 1, 1, 0, 0, 0, 0, 0)):
        args = [FAKE] * 12
        args[i] = NUL
        if not optional:
            assert lib.kda_block_norm_bwd(p, *args, FAKE, need, NUL) == _lib.KDA_ERR_INVALID
    assert lib.kda_block_norm_bwd(p, *[FAKE] * 12, FAKE, need - 1, NUL) == _lib.KDA_ERR_WORKSPACE


def test_norm_bindings_refuse():
    z, w = torch.zeros(4, 2, 64), torch.zeros(64)
    for args, kw, match in (((z, z, w), {}, "GPU"), ((z, z[:2], w), {}, "gate: expected"),
                            ((z, z.bfloat16(), w), {}, "gate: expected"),
                            ((z, z, w.bfloat16()), {}, "weight: expected"),
                            ((z.half(), z.half(), w), {}, "float32 or bfloat16"),
                            ((z, z, w), {"activation": "gelu"}, "activation")):
        with pytest.raises(KdaError, match=match):
            gated_norm(*args, **kw)
    x = torch.zeros(4, 64)
    for args, kw, match in (((x, x, w), {}, "GPU"), ((z, z, w), {}, "x: expected"),
                            ((x, x[:3], w), {}, "y: expected"),
                            ((x, x, w[:8]), {}, "w_pre: expected"),
                            ((x, x, w), {"w_post": x}, "w_post: expected"),
                            ((x, x, w), {"raw_gate": w}, "raw_gate: expected"),
                            ((x, x, w), {"raw_gate": x[:, :8]}, "raw_gate: expected")):
        with pytest.raises(KdaError, match=match):
            block_norm(*args, **kw)


# ------------------------------------------------------------------ short convolution


def sc(**kw):
    d = dict(n_seqs=2, total_tokens=9, C=64, W=4, dtype=_lib.KDA_BF16, activation=_lib.KDA_ACT_SILU,
             n_slots=4, x_stride=0)
    d.update(kw)
    return _lib.KdaShortConvProblem(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), _lib.KDA_ERR_INVALID),
    (dict(total_tokens=-1), _lib.KDA_ERR_INVALID),
    (dict(C=0), _lib.KDA_ERR_INVALID),
    (dict(C=60), _lib.KDA_ERR_UNSUPPORTED),
    (dict(C=(1 << 20) + 8), _lib.KDA_ERR_UNSUPPORTED),
    (dict(W=1), _lib.KDA_ERR_UNSUPPORTED),
    (dict(W=5), _lib.KDA_ERR_UNSUPPORTED),
    (dict(W=0), _lib.KDA_ERR_INVALID),
    (dict(dtype=2), _lib.KDA_ERR_UNSUPPORTED),
    (dict(activation=_lib.KDA_ACT_SIGMOID), _lib.KDA_ERR_UNSUPPORTED),
    (dict(x_stride=56), _lib.KDA_ERR_INVALID),
    (dict(x_stride=68), _lib.KDA_ERR_INVALID),
    (dict(C=1 << 20, total_tokens=1 << 20), _lib.KDA_ERR_UNSUPPORTED),
    (dict(total_tokens=0x7fffffff), _lib.KDA_ERR_UNSUPPORTED),
    (dict(n_seqs=1 << 26), _lib.KDA_ERR_UNSUPPORTED),
])
def test_short_conv_rejects(lib, kw, code):  # noqa: F811
    p = ctypes.byref(sc(**kw))
    assert lib.kda_short_conv_fwd(p, *[FAKE] * 7, NUL) == code
    assert lib.kda_short_conv_bwd(p, *[FAKE] * 11, FAKE, 1 << 40, NUL) == code
    assert lib.kda_short_conv_update(p, *[FAKE] * 7, NUL) == code
    assert lib.kda_short_conv_bwd_workspace_bytes(p) == 0


def test_short_conv_null_pointers_sequences_and_workspace(lib):  # noqa: F811
    p = ctypes.byref(sc())
    need = lib.kda_short_conv_bwd_workspace_bytes(p)
    for i, optional in enumerate((0, 0, 1, 0, 1, 0, 1)):  # x weight bias cu init y final
        args = [FAKE] * 7
        args[i] = NUL
        if not optional:  # without cu_seqlens there is one sequence
            assert lib.kda_short_conv_fwd(p, *args, NUL) == _lib.KDA_ERR_INVALID
    for i, optional in enumerate((0, 0, 1, 0, 1, 0, 1, 0, 0, 1, 1)):
        args = [FAKE] * 11
        args[i] = NUL
        if not optional:
            assert lib.kda_short_conv_bwd(p, *args, FAKE, need, NUL) == _lib.KDA_ERR_INVALID
    assert lib.kda_short_conv_bwd(p, *[FAKE] * 11, FAKE, need - 1, NUL) == _lib.KDA_ERR_WORKSPACE
    for i, optional in enumerate((0, 0, 1, 0, 1, 0, 0)):  # x weight bias cu idx state y
        args = [FAKE] * 7
        args[i] = NUL
        if not optional:  # without cu_seqlens there are as many sequences as tokens
            assert lib.kda_short_conv_update(p, *args, NUL) == _lib.KDA_ERR_INVALID
    few = ctypes.byref(sc(n_slots=1))
    assert lib.kda_short_conv_update(few, FAKE, FAKE, FAKE, FAKE, NUL, FAKE, FAKE, NUL) == _lib.KDA_ERR_INVALID
    none = ctypes.byref(sc(n_seqs=0, total_tokens=0))
    assert lib.kda_short_conv_update(none, *[NUL] * 7, NUL) == _lib.KDA_OK
    assert lib.kda_short_conv_fwd(none, NUL, NUL, NUL, FAKE, NUL, NUL, NUL, NUL) == _lib.KDA_OK


def test_short_conv_binding_refuses():
    x, w, b = torch.zeros(5, 64), torch.zeros(64, 4), torch.zeros(64)
    cu, st = torch.zeros(3, dtype=torch.int32), torch.zeros(2, 3, 64)
    for args, kw, match in (((x, w, b, cu), {}, "GPU"), ((x[0], w, b, cu), {}, "x: expected"),
                            ((x, w[:8], b, cu), {}, "weight: expected"),
                            ((x, w.bfloat16(), b, cu), {}, "weight: expected"),
                            ((x, w, b[:8], cu), {}, "bias: expected"),
                            ((x, w, b, cu.long()), {}, "cu_seqlens"),
                            ((x, w, b, cu), {"initial_state": st[:1]}, "initial_state: expected"),
                            ((x, w, b, cu), {"initial_state": st.bfloat16()}, "initial_state: expected"),
                            ((x.half(), w, b, cu), {}, "float32 or bfloat16"),
                            ((x, w, b, cu), {"activation": "relu"}, "activation")):
        with pytest.raises(KdaError, match=match):
            short_conv(*args, **kw)
    for args, kw, match in (((x, w, b, st), {}, "GPU"), ((x, w, b, st[0]), {}, "state: expected"),
                            ((x, w, b, st[:, :2]), {}, "state: expected"),
                            ((x, w, b, st.bfloat16()), {}, "state: expected"),
                            ((x, w, b, st), {"out": x[:4]}, "out: expected"),
                            ((x.clone().requires_grad_(True), w, b, st), {}, "not differentiable")):
        with pytest.raises(KdaError, match=match):
            short_conv_update(*args, **kw)


def test_gdn2_states_take_no_checkpoints(lib):  # noqa: F811
    from test_abi import good
    p = good()
    io = _lib.KdaStateIO()
    io.ckpt, io.ckpt_bytes = 0x2000, 1 << 40
    ws = ctypes.c_size_t(p.fwd_ws())
    assert lib.kda_gdn2_fwd_ex(p.ref, *[FAKE] * 10, ctypes.byref(io), FAKE, ws, NUL) == _lib.KDA_ERR_INVALID
    args = [FAKE] * 10
    args[4] = NUL
    assert lib.kda_gdn2_fwd_ex(p.ref, *args, None, FAKE, ws, NUL) == _lib.KDA_ERR_INVALID
    small = ctypes.c_size_t(p.fwd_ws() - 1)
    assert lib.kda_gdn2_fwd_ex(p.ref, *[FAKE] * 10, None, FAKE, small, NUL) == _lib.KDA_ERR_WORKSPACE


def test_sizes_that_are_not_built_are_named():
    x = rec_inputs(D=32)
    with pytest.raises(KdaError, match="K = 32, V = 32 are not built"):
        kda_recurrent(**x)
    z = torch.zeros(2, 96)
    with pytest.raises(KdaError, match="V = 96 is not built"):
        gated_norm(z, z, torch.zeros(96))
    for D in (12, 8200):
        z = torch.zeros(2, D)
        with pytest.raises(KdaError, match="D = %d is not built" % D):
            block_norm(z, z, torch.zeros(D))
    for C, W in ((12, 4), (16, 5), (16, 1), ((1 << 20) + 8, 2), (0, 4)):
        with pytest.raises(KdaError, match="not built"):
            short_conv(torch.zeros(1, C), torch.zeros(C, W))


def test_recurrent_refuses_a_per_head_gate_of_other_shape():
    with pytest.raises(KdaError, match="KDA_GATE_PER_HEAD takes"):
        kda_recurrent(**rec_inputs(), gate_mode=_lib.KDA_GATE_PER_HEAD)


# ------------------------------------------------------------------ overlap with the state


def at(addr):
    return ctypes.c_void_p(addr)


BASE = 1 << 32  # made-up addresses: every call below is refused before a launch


@pytest.mark.parametrize("g2", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_recurrent_refuses_a_state_over_its_other_tensors(lib, g2, per_head):  # noqa: F811
    if g2 and per_head:
        return
    N, T, H, K, slots, st = 3, 7, 2, 128, 5, 512  # bf16; q's rows 1024 bytes apart
    p = rec(total_tokens=T, n_slots=slots, q_stride=st,
            gate_mode=_lib.KDA_GATE_PER_HEAD if per_head else 0)
    row, head = T * H * K * 2, T * H * 2
    size = dict(q=((T - 1) * st + H * K) * 2, k=row, v=row, raw_g=head if per_head else row)
    size.update(dict(raw_b=row, raw_w=row) if g2 else dict(raw_beta=head))
    size.update(A_log=H * 4, dt_bias=H * 4 if per_head else H * K * 4, cu=(N + 1) * 4, idx=N * 4)
    state, fn = slots * H * K * K * 4, lib.kda_gdn2_recurrent if g2 else lib.kda_recurrent
    for name, n in dict(size, o=row).items():
        for addr in (BASE, BASE + state - 4, BASE - n + 2, BASE + 64):  # over either end, and inside
            where = {m: at((8 + 2 * i) * BASE) for i, m in enumerate(size)}
            o = at(6 * BASE)
            if name == "o":
                o = at(addr)
            else:
                where[name] = at(addr)
            got = fn(ctypes.byref(p), *where.values(), at(BASE), o, NUL)
            assert got == _lib.KDA_ERR_INVALID, (name, addr - BASE)


def test_short_conv_update_refuses_a_state_over_its_other_tensors(lib):  # noqa: F811
    N, T, C, W, slots, st = 3, 7, 64, 4, 5, 192
    p = sc(n_seqs=N, total_tokens=T, n_slots=slots, x_stride=st)
    size = dict(x=((T - 1) * st + C) * 2, weight=C * W * 4, bias=C * 4, cu=(N + 1) * 4, idx=N * 4)
    state = slots * (W - 1) * C * 2
    for name, n in dict(size, y=T * C * 2).items():
        for addr in (BASE, BASE + state - 2, BASE - n + 2, BASE + 64):
            where = {m: at((8 + 2 * i) * BASE) for i, m in enumerate(size)}
            y = at(6 * BASE)
            if name == "y":
                y = at(addr)
            else:
                where[name] = at(addr)
            got = lib.kda_short_conv_update(ctypes.byref(p), *where.values(), at(BASE), y, NUL)
            assert got == _lib.KDA_ERR_INVALID, (name, addr - BASE)


def test_more_indexed_sequences_than_the_slot_check_is_built_for(lib):  # noqa: F811
    # the check of slots named twice reads all earlier indices for every sequence
    n, cu = 65537, at(BASE)
    assert call_rec(lib, rec(n_seqs=n, total_tokens=9, H=1, n_slots=n), cu=cu, idx=FAKE) == _lib.KDA_ERR_UNSUPPORTED
    p = ctypes.byref(sc(n_seqs=n, total_tokens=9, n_slots=n))
    assert lib.kda_short_conv_update(p, FAKE, FAKE, FAKE, cu, FAKE, FAKE, FAKE, NUL) == _lib.KDA_ERR_UNSUPPORTED


def test_largest_launches_leave_room_for_the_rows_of_no_sequence(lib):  # noqa: F811
    n = (1 << 24) - 1
    p = rec(n_seqs=n, total_tokens=9, H=1, n_slots=n, zero_rest=1)
    assert call_rec(lib, p, cu=FAKE) == _lib.KDA_ERR_UNSUPPORTED
    p = ctypes.byref(sc(n_seqs=n, total_tokens=9, n_slots=n, zero_rest=1))
    assert lib.kda_short_conv_update(p, FAKE, FAKE, FAKE, FAKE, NUL, FAKE, FAKE, NUL) == _lib.KDA_ERR_UNSUPPORTED
