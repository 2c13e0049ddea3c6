"""The operators of a delta-rule layer run together as a model runs them
(needs an MI355X): short convolution, KDA, gated norm, an output projection,
block norm, in training against FP64 autograd of the same layer written out
in elementary torch operations on the host, and in decoding against the
packed forward.

Tolerances (fp32, normalised L2): each of the four operators is within 1e-5
of its definition forward and backward (their own tests); an error made in
one passes through at most the other three forward and the four backward, so
the layer's outputs and gradients are within 8e-5 as long as no operator
enlarges a relative error; the norms divide by what they are given and the
convolution and the delta rule are sums of comparable terms, for which 1e-4
is allowed.
"""
import numpy as np
import pytest
import torch

import kda_inputs
from oracle import layer_ref
from recompute_kda_chunked_amd import (block_norm, gated_norm, gdn2_forward, gdn2_recurrent, kda,
                                       kda_forward, kda_recurrent, short_conv, short_conv_update)
from test_gpu_states import announce, rel, to_np

pytestmark = pytest.mark.gpu

H, D, W = 2, 64, 4
M = 128  # model width


def weights(seed, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, sc=1.0, sh=0.0: (torch.randn(s, generator=gen) * sc + sh).to(device)  # noqa: E731
    return dict(proj=r(M, 3 * H * D, sc=M ** -0.5), gates=r(M, 2 * H * D + 8, sc=M ** -0.5),
                conv=r(3 * H * D, W, sc=0.5), conv_bias=r(3 * H * D, sc=0.1), A_log=r(H, sc=0.2),
                dt_bias=r(H, D, sc=0.3, sh=-2.0), norm=r(D, sc=0.2, sh=1.0),
                out=r(H * D, M, sc=(H * D) ** -0.5), w_post=r(M, sc=0.2, sh=1.0),
                w_pre=r(M, sc=0.2, sh=1.0), w_gate=r(M, M, sc=M ** -0.5))


def split(x, w):
    """Projections of the layer's input: q, k, v channels, and the raw gates
    (one product, its rows padded to a multiple of 16 bytes)."""
    g = x @ w["gates"]
    n = H * D
    return x @ w["proj"], g[:, :n].reshape(-1, H, D), g[:, n:2 * n].reshape(-1, H, D), g[:, 2 * n:2 * n + H]


def layer(x, res, w, cu, cu_host):
    """(residual stream, next block's input) of one layer on the packed tokens."""
    qkv, raw_g, gate, beta = split(x, w)
    c = short_conv(qkv, w["conv"], w["conv_bias"], cu)
    q, k, v = (c[:, i * H * D:(i + 1) * H * D].reshape(-1, H, D).contiguous() for i in range(3))
    o = kda(q, k, v, raw_g.contiguous(), beta.contiguous(), w["A_log"], w["dt_bias"], cu,
            cu_seqlens_host=cu_host, chunk=32)
    y = gated_norm(o, gate.contiguous(), w["norm"]).reshape(-1, H * D) @ w["out"]
    return block_norm(res, y, w["w_pre"], w_post=w["w_post"], raw_gate=x @ w["w_gate"],
                      residual_scale=0.5)


def layer_f64(x, res, w, cu):
    """The same written out, token by token."""
    qkv, raw_g, gate, beta = split(x, w)
    rms = lambda t, wt: t / torch.sqrt(torch.mean(t * t, -1, keepdim=True) + 1e-6) * wt  # noqa: E731
    l2 = lambda t: t / torch.sqrt(torch.sum(t * t, -1, keepdim=True) + 1e-6)  # noqa: E731
    rows = []
    for a, b in zip(cu[:-1], cu[1:]):
        e = torch.cat([qkv.new_zeros(W - 1, 3 * H * D), qkv[a:b]])
        S = qkv.new_zeros(H, D, D)
        for t in range(b - a):
            p = w["conv_bias"] + sum(w["conv"][:, j] * e[t + j] for j in range(W))
            q, k, v = (p * torch.sigmoid(p)).reshape(3, H, D)
            q, k, bt = l2(q), l2(k), torch.sigmoid(beta[a + t])[:, None]
            g = -5.0 * torch.sigmoid(torch.exp(w["A_log"])[:, None] * (raw_g[a + t] + w["dt_bias"]))
            S = S * torch.exp(g)[:, :, None]
            S = S + k[:, :, None] * (bt * (v - torch.sum(S * k[:, :, None], 1)))[:, None, :]
            rows.append(torch.sum(S * q[:, :, None], 1))
    o = torch.stack(rows)
    y = (rms(o, w["norm"]) * torch.sigmoid(gate)).reshape(-1, H * D) @ w["out"]
    out = res + 0.5 * torch.sigmoid(x @ w["w_gate"]) * rms(y, w["w_post"])
    return out, rms(out, w["w_pre"])


def test_training_step_of_two_layers():
    announce("two layers, forward and backward")
    cu = [0, 20, 20, 27, 61]
    T = cu[-1]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(5)
    x0, res0, d0, d1 = (torch.randn(T, M, generator=gen) for _ in range(4))
    results = []
    for dev, dt in (("cuda", torch.float32), ("cpu", torch.float64)):
        ws = [{k: t.to(dev, dt).requires_grad_(True) for k, t in weights(s, "cpu").items()} for s in (1, 2)]
        x, res = (t.to(dev, dt).requires_grad_(True) for t in (x0, res0))
        r, h = res, x
        for w in ws:
            r, h = layer(h, r, w, cud, cu) if dev == "cuda" else layer_f64(h, r, w, cu)
        leaves = [x, res] + [t for w in ws for t in w.values()]
        grads = torch.autograd.grad((r, h), leaves, (d0.to(dev, dt), d1.to(dev, dt)))
        results.append([to_np(t) for t in (r, h, *grads)])
    names = ["r", "h", "dx", "dres"] + ["d%s%d" % (k, i) for i in (0, 1) for k in weights(1, "cpu")]
    errs = {n: rel(a, b) for n, a, b in zip(names, *results)}
    print(" ".join("%s=%.1e" % kv for kv in errs.items()), flush=True)
    assert all(np.isfinite(e) and e <= 1e-4 for e in errs.values()), errs


def test_prompt_then_captured_decoding():
    announce("prompts packed, then tokens one by one from a graph")
    w = weights(3)
    lens, more = [30, 1, 17], 4
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n + more)
    gen = torch.Generator().manual_seed(6)
    x, res = (torch.randn(cu[-1], M, generator=gen).cuda() for _ in range(2))
    with torch.no_grad():
        want = layer(x, res, w, torch.tensor(cu, dtype=torch.int32, device="cuda"), cu)
        # the prompts alone, leaving both states
        rows = torch.cat([torch.arange(a, a + n) for a, n in zip(cu, lens)]).cuda()
        pcu = [0, 30, 31, 48]
        pcud = torch.tensor(pcu, dtype=torch.int32, device="cuda")
        qkv, raw_g, _, beta = split(x[rows], w)
        c, conv_state = short_conv(qkv, w["conv"], w["conv_bias"], pcud, output_final_state=True)
        q, k, v = (c[:, i * H * D:(i + 1) * H * D].reshape(-1, H, D).contiguous() for i in range(3))
        _, ht, _ = kda_forward(q, k, v, raw_g.contiguous(), beta.contiguous(), w["A_log"], w["dt_bias"],
                               pcud, cu_seqlens_host=pcu, chunk=32, output_final_state=True)
        # pools with room, a batch padded to four sequences
        slots = torch.tensor([4, 0, 2, -1], dtype=torch.int32, device="cuda")
        pool, conv_pool = torch.zeros(5, H, D, D, device="cuda"), torch.zeros(5, W - 1, 3 * H * D, device="cuda")
        pool[slots[:3].long()], conv_pool[slots[:3].long()] = ht, conv_state
        xt, rt = torch.zeros(4, M, device="cuda"), torch.zeros(4, M, device="cuda")

        def step():
            qkv, raw_g, gate, beta = split(xt, w)
            c = short_conv_update(qkv, w["conv"], w["conv_bias"], conv_pool, state_indices=slots)
            q, k, v = (c[:, i * H * D:(i + 1) * H * D].view(4, H, D) for i in range(3))
            o = kda_recurrent(q, k, v, raw_g, beta, w["A_log"], w["dt_bias"], pool, state_indices=slots)
            y = gated_norm(o, gate.contiguous(), w["norm"]).view(4, H * D) @ w["out"]
            return block_norm(rt, y, w["w_pre"], w_post=w["w_post"], raw_gate=xt @ w["w_gate"],
                              residual_scale=0.5)

        keep = pool.clone(), conv_pool.clone()
        step()  # warm up, then put the states back
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        pool.copy_(keep[0])
        conv_pool.copy_(keep[1])
        for j in range(more):
            at = torch.tensor([a + n + j for a, n in zip(cu, lens)], device="cuda")
            xt[:3], rt[:3] = x[at], res[at]
            graph.replay()
            torch.cuda.synchronize()
            for got, ref in zip(out, want):
                assert rel(to_np(got[:3]), to_np(ref[at])) <= 1e-4, j
                assert bool(torch.isfinite(got).all())
        assert bool((pool[[1, 3]] == 0).all()) and bool((conv_pool[[1, 3]] == 0).all())


@pytest.mark.parametrize("dtype,Dh,chunk", [(torch.float32, 128, 32), (torch.bfloat16, 64, 64)])
def test_gdn2_prompt_then_decoding(dtype, Dh, chunk):
    announce("GDN-2 prompt with states, then tokens %s" % dtype)
    lens, more = [70, 0, 9], 3
    x = kda_inputs.make_inputs(lens, H, Dh, Dh, dtype, 8, "cuda", dt_bias=-1.0, gdn2=True)
    y = kda_inputs.make_inputs([more] * 3, H, Dh, Dh, dtype, 9, "cuda", dt_bias=-1.0, gdn2=True)
    h0 = kda_inputs.make_states(3, H, Dh, Dh, 10, "cuda")["h0"]
    names = ("q", "k", "v", "raw_g", "raw_b", "raw_w", "A_log", "dt_bias")
    kw = dict(cu_seqlens_host=x["cu_seqlens_host"], chunk=chunk)
    o, ht = gdn2_forward(*[x[n] for n in names], x["cu_seqlens"], initial_state=h0, output_final_state=True, **kw)
    ref = lambda z, s: layer_ref.recurrent(z["q"], z["k"], z["v"], z["raw_g"], z["A_log"], z["dt_bias"], s,  # noqa: E731
                                           z["cu_seqlens_host"], raw_b=z["raw_b"], raw_w=z["raw_w"])
    ro, rs = ref(x, h0)
    tol = 1e-5 if dtype is torch.float32 else 5e-3  # the chunked form's tolerances
    assert rel(to_np(o), ro) <= tol and rel(to_np(ht), rs) <= tol
    assert torch.equal(ht[1], h0[1])
    zero = gdn2_forward(*[x[n] for n in names], x["cu_seqlens"], initial_state=torch.zeros_like(h0), **kw)
    assert torch.equal(zero, gdn2_forward(*[x[n] for n in names], x["cu_seqlens"], **kw))
    ro, rs = ref(y, ht)
    o = gdn2_recurrent(*[y[n] for n in names], ht, y["cu_seqlens"])
    assert rel(to_np(ht), rs) <= 1e-5
    assert rel(to_np(o), ro) <= 1e-5 + (0 if dtype is torch.float32 else 2.0 ** -8)


def tiled(seed, *shape):
    """bf16 values of a shape of more than 2^31 elements: one random block
    repeated."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = int(np.prod(shape))
    block = torch.randn(1 << 20, generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    whole = n >> 20
    out[:whole << 20].view(whole, 1 << 20).copy_(block.expand(whole, 1 << 20))
    out[whole << 20:] = block[:n - (whole << 20)]
    return out.view(shape)


def test_norms_past_32_bit_offsets():
    announce("norms of more than 2^31 elements")
    from recompute_kda_chunked_amd import (block_norm_backward, block_norm_forward, gated_norm_backward,
                                           gated_norm_forward)
    rows = (1 << 24) + 77
    o, g, dy = (tiled(s, rows, 128) for s in (1, 2, 3))
    w = torch.linspace(0.5, 1.5, 128, device="cuda")
    y = gated_norm_forward(o, g, w)
    do, dg, _ = gated_norm_backward(o, g, w, dy)
    e = slice(rows - 300, rows)
    part = gated_norm_backward(o[e], g[e], w, dy[e])
    assert torch.equal(y[e], gated_norm_forward(o[e], g[e], w))
    assert torch.equal(do[e], part[0]) and torch.equal(dg[e], part[1])
    del o, g, dy, y, do, dg
    T, D = (1 << 18) + 9, 8192
    x, y, d0, d1 = (tiled(s, T, D) for s in (4, 5, 6, 7))
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    out = block_norm_forward(x, y, w, w_post=w)
    got = block_norm_backward(x, y, w, d0, d1, w_post=w)
    e = slice(T - 20, T)
    assert all(torch.equal(a[e], b) for a, b in zip(out, block_norm_forward(x[e], y[e], w, w_post=w)))
    part = block_norm_backward(x[e], y[e], w, d0[e], d1[e], w_post=w)
    assert torch.equal(got[0][e], part[0]) and torch.equal(got[1][e], part[1])


def test_convolution_past_32_bit_offsets():
    announce("convolution of more than 2^31 elements")
    from recompute_kda_chunked_amd import short_conv_backward, short_conv_forward
    T, C = (1 << 18) + 21, 8192
    x, dy = tiled(8, T, C), tiled(9, T, C)
    w, b = torch.randn(C, W, device="cuda") * 0.5, torch.randn(C, device="cuda")
    cu = torch.tensor([0, T - 50, T], dtype=torch.int32, device="cuda")
    y, final = short_conv_forward(x, w, b, cu, output_final_state=True)
    dx = short_conv_backward(x, w, b, dy, cu)[0]
    e = slice(T - 50, T)
    ye, fe = short_conv_forward(x[e], w, b, output_final_state=True)
    assert torch.equal(y[e], ye) and torch.equal(final[1:], fe)
    assert torch.equal(dx[e], short_conv_backward(x[e], w, b, dy[e])[0])


def test_launches_are_timed_by_kind():
    announce("profile kinds")
    from recompute_kda_chunked_amd import _lib
    o = torch.randn(5, 2, 64, device="cuda").requires_grad_(True)
    w, x = torch.ones(64, device="cuda"), torch.randn(5, 64, device="cuda").requires_grad_(True)
    cw, cb = torch.randn(64, W, device="cuda"), torch.randn(64, device="cuda")
    state = torch.zeros(5, 2, 64, 64, device="cuda")
    z = o.detach()
    _lib.profile_begin()
    out = (gated_norm(o, z, w), *block_norm(x, x.detach(), w), short_conv(x, cw, cb))
    grads = torch.autograd.grad(out, (o, x), out)
    short_conv_update(x.detach(), cw, cb, torch.zeros(5, W - 1, 64, device="cuda"))
    kda_recurrent(z, z, z, z, z[:, :, 0].contiguous(), torch.zeros(2, device="cuda"),
                  torch.zeros(2, 64, device="cuda"), state)
    prof = _lib.profile_end()
    assert len(grads) == 2
    # the backward calls are made by autograd's own thread: their launches are not this thread's
    for kind in ("gated_norm", "block_norm", "short_conv", "short_conv_update", "recurrent"):
        assert prof[kind][0] == 1 and prof[kind][1] > 0, kind
    assert prof["recurrent"][2] == 10 and prof["gated_norm"][2] == 10 and prof["block_norm"][2] == 5
