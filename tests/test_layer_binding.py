"""The binding of the operators around the chunked one as torch sees it,
without a GPU: the launch is left out and host tensors are let through, so
that what autograd and its neighbours make of a call can be looked at."""
import pytest
import torch
from torch.autograd import forward_ad

from recompute_kda_chunked_amd import (KdaError, block_norm, gated_norm, gdn2_recurrent,
                                       kda_recurrent, layer, ops, short_conv, short_conv_update)
from test_layer_host import rec_inputs


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setattr(layer, "_dev", lambda t, name: t.device)
    monkeypatch.setattr(layer, "_call", lambda *args, **kw: None)


def gdn2_inputs():
    x = rec_inputs()
    beta = x.pop("raw_beta")
    return dict(x, raw_b=torch.zeros_like(x["k"]), raw_w=torch.zeros(*beta.shape, 64))


def conv_update_inputs():
    return dict(x=torch.zeros(5, 64), weight=torch.zeros(64, 4), bias=torch.zeros(64),
                state=torch.zeros(5, 3, 64))


DIFFERENTIABLE = [
    (gated_norm, lambda: dict(o=torch.zeros(4, 2, 64), gate=torch.zeros(4, 2, 64), weight=torch.zeros(64))),
    (block_norm, lambda: dict(x=torch.zeros(4, 64), y=torch.zeros(4, 64), w_pre=torch.zeros(64),
                              w_post=torch.zeros(64), raw_gate=torch.zeros(4))),
    (short_conv, lambda: dict(x=torch.zeros(5, 64), weight=torch.zeros(64, 4), bias=torch.zeros(64),
                              initial_state=torch.zeros(1, 3, 64))),
]
IN_PLACE = [(kda_recurrent, rec_inputs), (gdn2_recurrent, gdn2_inputs), (short_conv_update, conv_update_inputs)]


@pytest.mark.parametrize("fn,make", DIFFERENTIABLE)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused_by_the_autograd_functions(fn, make, grad):
    for name in make():
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            x = make()
            fn(**x)  # a level without tangents changes nothing
            x[name] = forward_ad.make_dual(x[name], torch.ones_like(x[name]))
            with pytest.raises(NotImplementedError, match="jvp"):
                fn(**x)


@pytest.mark.parametrize("fn,make", IN_PLACE)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused_by_the_decoding_forms(fn, make, grad):
    for name in make():
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            x = make()
            fn(**x)
            x[name] = forward_ad.make_dual(x[name], torch.ones_like(x[name]))
            with pytest.raises(KdaError, match="not differentiable"):
                fn(**x)


@pytest.mark.parametrize("fn,make", DIFFERENTIABLE)
def test_a_trace_keeps_the_call(fn, make, monkeypatch):
    names, calls = list(make()), []
    monkeypatch.setattr(layer, "_call", lambda dev, name, *args, **kw: calls.append(name))
    traced = torch.jit.trace(lambda *t: fn(**dict(zip(names, t))), tuple(make().values()), check_trace=False)
    assert any(n.kind() == "prim::PythonOp" for n in traced.graph.nodes()) and len(calls) == 1
    traced(*make().values())
    assert len(calls) == 2


@pytest.mark.parametrize("fn,make", IN_PLACE)
def test_decoding_forms_refuse_a_trace(fn, make):
    names = list(make())
    with pytest.raises(KdaError, match="cannot be traced"):
        torch.jit.trace(lambda *t: fn(**dict(zip(names, t))), tuple(make().values()), check_trace=False)


@pytest.mark.parametrize("fn,make", IN_PLACE)
def test_autograd_sees_what_a_call_overwrites(fn, make):
    for name in ("state", "out"):
        x = make()
        if name == "out":
            x["out"] = fn(**x)
        w = torch.ones((), requires_grad=True)
        loss = (w * x[name]).sum()  # keeps state or out for its backward
        version = x[name]._version
        fn(**x)
        assert x[name]._version > version
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():  # tensors without versions
        x = make()
        fn(**x, out=fn(**x))
    fn(**x)


@pytest.mark.parametrize("fn,make", IN_PLACE)
def test_inputs_keep_their_versions(fn, make):
    x = make()
    versions = {n: t._version for n, t in x.items()}
    fn(**x)
    assert all(t._version == versions[n] for n, t in x.items() if n != "state")


@pytest.mark.parametrize("fn,make", IN_PLACE)
def test_an_out_that_requires_a_gradient_is_refused(fn, make):
    x = make()
    out = fn(**x).requires_grad_(True)
    with pytest.raises(KdaError, match="not differentiable"):
        fn(**x, out=out)
    with pytest.raises(KdaError, match="not differentiable"):
        fn(**x, out=out * 1)
    with torch.no_grad():
        assert fn(**x, out=out) is out
    with forward_ad.dual_level(), pytest.raises(KdaError, match="not differentiable"):
        fn(**x, out=forward_ad.make_dual(out.detach(), torch.ones_like(out)))


def test_too_many_indexed_sequences_are_named():
    n = 65537
    idx, cu = torch.zeros(n, dtype=torch.int32), torch.zeros(n + 1, dtype=torch.int32)
    for fn, make in IN_PLACE:
        with pytest.raises(KdaError, match="more than 65536"):
            fn(**make(), cu_seqlens=cu, state_indices=idx)
        fn(**make(), cu_seqlens=cu[:n], state_indices=idx[:n - 1])


def test_an_out_that_the_chunked_forward_cannot_fill_is_refused():
    good = torch.empty(6, 2, 64)
    ops._check_out(good, 6, 2, 64, torch.float32, good.device)
    ops._check_out(good.view(6, 128), 6, 2, 64, torch.float32, good.device)
    for bad, match in ((good[:5], "out: expected"), (good.bfloat16(), "out: expected"),
                       (torch.empty(6, 2, 128), "out: expected"), (torch.empty(6, 2, 128)[..., :64], "contiguous"),
                       (torch.empty(6 * 128 + 1)[1:].view(6, 2, 64), "aligned"),
                       (good.to("meta"), "on cpu")):
        with pytest.raises(KdaError, match=match):
            ops._check_out(bad, 6, 2, 64, torch.float32, good.device)
