"""Cases for measuring the operators around the chunked delta rule: the recurrent (decoding) form
of KDA and GDN-2, the gated output norm, the norms around a block with its gate and residual
scale, and the short causal convolution with its decoding state.

``own`` selects the framework's kernels; otherwise ``run`` computes the same with elementary
torch operations in fp32 (gradients by torch's autograd). ``exact`` computes it in fp64 from the
definitions, with hand-written gradients.
"""
from __future__ import annotations

import math
import random

import torch

own = False

F32, BF16 = "float32", "bfloat16"


# ---------------------------------------------------------------------------- cases


def listed():
    return [
        # one user's decoding step at a small model's head count: latency alone counts
        _rec("kda_recurrent", "kda_step_1x8x64_f32", F32, n=1, H=8, D=64, L=1),
        # a decoding batch of a KDA layer, states scattered over a larger pool
        _rec("kda_recurrent", "kda_step_64x32x128_bf16", BF16, n=64, H=32, D=128, L=1),
        # a large decoding batch with one gate per head, padded to a fixed launch size
        _rec("kda_recurrent", "kda_step_251x32x128_bf16_head", BF16, n=251, H=32, D=128, L=1,
             gate="head", pad=5),
        # ragged runs of up to 8 drafted tokens a sequence, some sequences with none
        _rec("kda_recurrent", "kda_draft_37x64x128_bf16", BF16, n=37, H=64, D=128, L=8),
        # GDN-2 decoding: a batch of single tokens, and short ragged runs in fp32
        _rec("gdn2_recurrent", "gdn2_step_128x16x128_bf16", BF16, n=128, H=16, D=128, L=1),
        _rec("gdn2_recurrent", "gdn2_draft_9x12x64_f32", F32, n=9, H=12, D=64, L=5),
        # the output norm of one decoding batch, and of a training step at 8K tokens x 64 heads
        _gn("gated_norm_16x32x128_bf16", BF16, T=16, H=32, V=128, act="sigmoid", train=False),
        _gn("gated_norm_8192x64x128_bf16_train", BF16, T=8192, H=64, V=128, act="sigmoid",
            train=True),
        # between two blocks: an odd fp32 batch with a gate per token, and a training step
        _bn("block_norm_131x2560_f32", F32, T=131, D=2560, gate="token", post=True, train=False),
        _bn("block_norm_8191x4096_bf16_train", BF16, T=8191, D=4096, gate="channel", post=True,
            train=True),
        # the convolution of fused q, k, v channels for a decoding batch, and a packed training
        # batch of one of them
        _cv("short_conv_update_64x12288_bf16", BF16, T=64, C=12288, W=4, n=64, mode="update"),
        _cv("short_conv_8192x8192_bf16_train", BF16, T=8192, C=8192, W=4, n=7, mode="train"),
    ]


def _rec(op, name, dtype, n, H, D, L, gate="channel", pad=0):
    c = {"op": op, "dtype": dtype, "n": n, "H": H, "D": D, "L": L, "gate": gate, "pad": pad}
    return dict(c, name=name) if name else c


def _gn(name, dtype, T, H, V, act, train):
    c = {"op": "gated_norm", "dtype": dtype, "T": T, "H": H, "V": V, "act": act, "train": train}
    return dict(c, name=name) if name else c


def _bn(name, dtype, T, D, gate, post, train):
    c = {"op": "block_norm", "dtype": dtype, "T": T, "D": D, "gate": gate, "post": post,
         "train": train}
    return dict(c, name=name) if name else c


def _cv(name, dtype, T, C, W, n, mode, act="silu", bias=True):
    c = {"op": "short_conv", "dtype": dtype, "T": T, "C": C, "W": W, "n": n, "mode": mode,
         "act": act, "bias": bias}
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["kda_recurrent", "kda_recurrent", "gdn2_recurrent", "gated_norm",
                     "block_norm", "short_conv"])
    dtype = rng.choice([F32, BF16])
    if op in ("kda_recurrent", "gdn2_recurrent"):
        D, H, L = rng.choice([64, 128]), _spread(rng, 1, 64), rng.choice([1, 1, _spread(rng, 2, 16)])
        room = 251 * 32 * 128 * 128 // (H * D * D * max(1, L // 3))
        n = _spread(rng, 1, max(1, min(256, room)))
        gate = rng.choice(["channel", "head"]) if op == "kda_recurrent" else "channel"
        return _rec(op, None, dtype, n, H, D, L, gate, rng.choice([0, 0, rng.randint(1, 4)]))
    if op == "gated_norm":
        V, H = rng.choice([64, 128, 256]), _spread(rng, 1, 64)
        T = _spread(rng, 1, min(16384, (1 << 25) // (H * V)))
        return _gn(None, dtype, T, H, V, rng.choice(["sigmoid", "silu"]), rng.random() < 0.6)
    if op == "block_norm":
        D = 8 * _spread(rng, 8, 1024)
        T = _spread(rng, 1, min(16384, (1 << 24) // D))
        return _bn(None, dtype, T, D, rng.choice(["none", "token", "channel"]),
                   rng.random() < 0.7, rng.random() < 0.6)
    mode, C, W = rng.choice(["fwd", "train", "update"]), 8 * _spread(rng, 8, 1536), rng.randint(2, 4)
    n = _spread(rng, 1, 512 if mode == "update" else 24)
    T = n * rng.choice([1, 1, 2, 5]) if mode == "update" else _spread(rng, 1, min(16384, (1 << 25) // C))
    return _cv(None, dtype, T, C, W, n, mode, rng.choice(["silu", "silu", "none"]),
               rng.random() < 0.5)


def _lens(case):
    """Tokens of each sequence, the same for every seed: of a recurrent case (up to L each, the
    first one L, some of them none), of a convolution case (T tokens cut at random places)."""
    r = random.Random("%s %s" % (case["n"], case.get("L", case.get("T"))))
    if "L" in case:
        return [case["L"]] + [case["L"] if case["L"] == 1 else r.randint(0, case["L"])
                              for _ in range(case["n"] - 1)]
    n, T = case["n"], case["T"]
    if case["mode"] == "update":
        return [T // n] * n
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    op = case["op"]
    if op in ("kda_recurrent", "gdn2_recurrent"):
        H, D, rows = case["H"], case["D"], sum(_lens(case))
        gates = (D if case["gate"] == "channel" else 1) + (1 if op == "kda_recurrent" else 2 * D)
        return {"bytes": case["n"] * H * D * D * 8 + rows * H * (4 * D + gates) * e,
                "flops": rows * H * 7 * D * D}
    if op == "gated_norm":
        n = case["T"] * case["H"] * case["V"]
        return {"bytes": (6 if case["train"] else 3) * n * e, "flops": (30 if case["train"] else 10) * n}
    if op == "block_norm":
        n, t = case["T"] * case["D"], case["train"]
        per = (8 if t else 4) + (0 if case["gate"] != "channel" else 2 if t else 1)
        return {"bytes": per * n * e, "flops": (40 if t else 15) * n}
    n, W = case["T"] * case["C"], case["W"]
    if case["mode"] == "update":
        return {"bytes": 2 * n * e + 2 * case["n"] * (W - 1) * case["C"] * e, "flops": n * (2 * W + 6)}
    return {"bytes": (4 if case["mode"] == "train" else 2) * n * e,
            "flops": n * ((6 * W + 20) if case["mode"] == "train" else (2 * W + 6))}


# ---------------------------------------------------------------------------- inputs


class State:
    """What a user's program holds before the call."""


def prepare(case, seed):
    s = State()
    s.case = dict(case)
    s.dtype = getattr(torch, case["dtype"])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype=None, scale=1.0, shift=0.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(scale).add_(shift).to(dtype or s.dtype)

    op = case["op"]
    if op in ("kda_recurrent", "gdn2_recurrent"):
        _prepare_recurrent(s, case, gen, randn)
    elif op == "gated_norm":
        T, H, V = case["T"], case["H"], case["V"]
        s.o, s.gate = randn(T, H, V, scale=0.7), randn(T, H, V)
        s.weight = randn(V, dtype=torch.float32, scale=0.2, shift=1.0)
        s.dy = randn(T, H, V) if case["train"] else None
        s.leaves = (s.o, s.gate, s.weight)
    elif op == "block_norm":
        T, D = case["T"], case["D"]
        s.x, s.y = randn(T, D, scale=2.0), randn(T, D)
        s.w_pre = randn(D, dtype=torch.float32, scale=0.2, shift=1.0)
        s.w_post = randn(D, dtype=torch.float32, scale=0.2, shift=1.0) if case["post"] else None
        s.gate = {"none": lambda: None, "token": lambda: randn(T), "channel": lambda: randn(T, D)}[case["gate"]]()
        s.scale = 0.22
        s.dx_out, s.dh = (randn(T, D), randn(T, D)) if case["train"] else (None, None)
        s.leaves = tuple(t for t in (s.x, s.y, s.w_pre, s.w_post, s.gate) if t is not None)
    else:
        T, C, W, n = case["T"], case["C"], case["W"], case["n"]
        s.x = randn(T, C)
        s.weight = randn(C, W, dtype=torch.float32, scale=0.5)
        s.bias = randn(C, dtype=torch.float32, scale=0.2) if case["bias"] else None
        lens = _lens(case)
        s.cu = _cu(lens)
        if case["mode"] == "update":
            s.pool = randn(n + n // 4 + 1, W - 1, C)
            s.slots = torch.randperm(s.pool.shape[0], generator=gen, device="cuda")[:n].to(torch.int32)
            if T == n:
                s.cu = None  # one token a sequence
        else:
            s.init = randn(n, W - 1, C)
            s.dy, s.dfinal = (randn(T, C), randn(n, W - 1, C)) if case["mode"] == "train" else (None, None)
            s.leaves = tuple(t for t in (s.x, s.weight, s.bias, s.init) if t is not None)
        # where each tap of each token, and each row of the state left behind, lies among the
        # states' rows followed by the tokens' rows
        s.taps, s.left = _tap_rows(lens, W)
    if case.get("train") or case.get("mode") == "train":
        for t in s.leaves:
            t.requires_grad_(True)
    return s


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _prepare_recurrent(s, case, gen, randn):
    n, H, D, L, pad = case["n"], case["H"], case["D"], case["L"], case["pad"]
    lens = _lens(case)
    rows = sum(lens)
    T = rows + pad if L == 1 else rows  # padded sequences have one token each, or none
    g = (T, H) if case["gate"] == "head" else (T, H, D)
    s.q, s.k, s.v, s.raw_g = randn(T, H, D), randn(T, H, D), randn(T, H, D), randn(*g)
    if case["op"] == "kda_recurrent":
        s.raw_beta = randn(T, H)
    else:
        s.raw_b, s.raw_w = randn(T, H, D), randn(T, H, D)
    s.A_log = randn(H, dtype=torch.float32, scale=0.3)
    s.dt_bias = randn(*g[1:], dtype=torch.float32, scale=0.5, shift=-2.0)
    slots = n + n // 4 + 1
    s.pool = randn(slots, H, D, D, dtype=torch.float32, scale=0.3)
    s.slots = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
    if pad:  # a batch filled up to its launch size: no state behind the last ones
        s.slots = torch.cat([s.slots, torch.full((pad,), -1, dtype=torch.int32, device="cuda")])
    s.cu = None if L == 1 else _cu(lens + [0] * pad)
    s.live = n
    # row of the j-th token of each sequence; T (a row of padding) where it has none
    first = [sum(lens[:i]) for i in range(n)]
    s.steps = torch.tensor([[first[i] + j if j < lens[i] else T for i in range(n)]
                            for j in range(L)], device="cuda")


def _tap_rows(lens, W):
    n, taps, left, t0 = len(lens), [], [], 0
    for i, m in enumerate(lens):
        at = [i * (W - 1) + j for j in range(W - 1)] + [n * (W - 1) + t0 + t for t in range(m)]
        taps += [at[t:t + W] for t in range(m)]
        left += at[m:]
        t0 += m
    return (torch.tensor(taps, device="cuda").reshape(-1, W).t().contiguous(),
            torch.tensor(left, device="cuda"))


# ---------------------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    op = s.case["op"]
    if op in ("kda_recurrent", "gdn2_recurrent"):
        return _plain_recurrent(s)
    if op == "gated_norm":
        y = _plain_gated_norm(s)
        if not s.case["train"]:
            return y
        return (y.detach(), *torch.autograd.grad(y, s.leaves, s.dy))
    if op == "block_norm":
        out = _plain_block_norm(s)
        if not s.case["train"]:
            return out
        return (*[t.detach() for t in out], *torch.autograd.grad(out, s.leaves, (s.dx_out, s.dh)))
    if s.case["mode"] == "update":
        state = s.pool.index_select(0, s.slots)
        y, state = _plain_conv(s, state)
        s.pool.index_copy_(0, s.slots.long(), state)
        return y, s.pool
    y, final = _plain_conv(s, s.init)
    if s.case["mode"] == "fwd":
        return y, final
    return (y.detach(), final.detach(), *torch.autograd.grad((y, final), s.leaves, (s.dy, s.dfinal)))


def _run_own(s):
    import recompute_kda_chunked_amd as kda
    c, op = s.case, s.case["op"]
    if op == "kda_recurrent":
        o = kda.kda_recurrent(s.q, s.k, s.v, s.raw_g, s.raw_beta, s.A_log, s.dt_bias, s.pool, s.cu,
                              state_indices=s.slots)
        return o, s.pool
    if op == "gdn2_recurrent":
        o = kda.gdn2_recurrent(s.q, s.k, s.v, s.raw_g, s.raw_b, s.raw_w, s.A_log, s.dt_bias,
                               s.pool, s.cu, state_indices=s.slots)
        return o, s.pool
    if op == "gated_norm":
        y = kda.gated_norm(s.o, s.gate, s.weight, activation=c["act"])
        if not c["train"]:
            return y
        return (y.detach(), *torch.autograd.grad(y, s.leaves, s.dy))
    if op == "block_norm":
        out = kda.block_norm(s.x, s.y, s.w_pre, w_post=s.w_post, raw_gate=s.gate,
                             residual_scale=s.scale)
        if not c["train"]:
            return out
        return (*[t.detach() for t in out], *torch.autograd.grad(out, s.leaves, (s.dx_out, s.dh)))
    if c["mode"] == "update":
        y = kda.short_conv_update(s.x, s.weight, s.bias, s.pool, s.cu, state_indices=s.slots,
                                  activation=c["act"])
        return y, s.pool
    y, final = kda.short_conv(s.x, s.weight, s.bias, s.cu, initial_state=s.init,
                              output_final_state=True, activation=c["act"])
    if c["mode"] == "fwd":
        return y, final
    return (y.detach(), final.detach(), *torch.autograd.grad((y, final), s.leaves, (s.dy, s.dfinal)))


# ---------------------------------------------------------------------------- plain forms


def _plain_recurrent(s):
    c = s.case
    q, k, v = s.q.float(), s.k.float(), s.v.float()
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    z = (s.raw_g.float() + s.dt_bias) * (torch.exp(s.A_log) if c["gate"] == "head" else torch.exp(s.A_log)[:, None])
    decay = torch.exp(-5.0 * torch.sigmoid(z))
    decay = decay[..., None] if c["gate"] == "head" else decay
    if c["op"] == "kda_recurrent":
        beta = torch.sigmoid(s.raw_beta.float())[..., None]
        erase, write = beta * k, beta * v
    else:
        erase, write = torch.sigmoid(s.raw_b.float()) * k, torch.sigmoid(s.raw_w.float()) * v
    state = s.pool.index_select(0, s.slots[:s.live])
    if c["L"] == 1:
        n = s.live
        o, state = _plain_step(state, q[:n], k[:n], erase[:n], write[:n], decay[:n])
        out = torch.zeros_like(s.v)
        out[:n] = o.to(s.dtype)
    else:
        def padded(x, value=0.0):
            return torch.cat([x, x.new_full((1, *x.shape[1:]), value)])

        q, k, erase, write, decay = padded(q), padded(k), padded(erase), padded(write), padded(decay, 1.0)
        out = torch.zeros((s.v.shape[0] + 1, *s.v.shape[1:]), dtype=s.dtype, device=s.v.device)
        for at in s.steps:
            o, state = _plain_step(state, q[at], k[at], erase[at], write[at], decay[at])
            out[at] = o.to(s.dtype)
        out = out[:-1]
    s.pool.index_copy_(0, s.slots[:s.live].long(), state)
    return out, s.pool


def _plain_step(state, q, k, erase, write, decay):
    """One token of every sequence: states [n, H, K, V], rows [n, H, K or V]."""
    state = state * decay[..., None]
    write = write - torch.matmul(erase[..., None, :], state)[..., 0, :]
    state = state + k[..., None] * write[..., None, :]
    return torch.matmul(q[..., None, :], state)[..., 0, :], state


def _plain_gated_norm(s):
    o, g = s.o.float(), s.gate.float()
    n = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-6)
    a = torch.sigmoid(g)
    a = g * a if s.case["act"] == "silu" else a
    return (n * s.weight * a).to(s.dtype)


def _plain_block_norm(s):
    z = s.y.float()
    if s.w_post is not None:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s.w_post
    if s.gate is not None:
        a = torch.sigmoid(s.gate.float())
        z = z * (a if s.case["gate"] == "channel" else a[:, None])
    x = s.x.float() + s.scale * z
    h = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s.w_pre
    return x.to(s.dtype), h.to(s.dtype)


def _plain_conv(s, state):
    rows = torch.cat([state.float().reshape(-1, s.case["C"]), s.x.float()])
    p = sum(rows.index_select(0, at) * s.weight[:, j] for j, at in enumerate(s.taps))
    p = p if s.bias is None else p + s.bias
    y = p * torch.sigmoid(p) if s.case["act"] == "silu" else p
    final = rows.index_select(0, s.left).reshape(state.shape)
    return y.to(s.dtype), final.to(s.dtype)


# ---------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] in ("kda_recurrent", "gdn2_recurrent"):
            return _exact_recurrent(s)
        if case["op"] == "gated_norm":
            return _exact_gated_norm(s)
        if case["op"] == "block_norm":
            return _exact_block_norm(s)
        return _exact_conv(s)


def _exact_recurrent(s):
    """S_t = (I - kh e^T) Diag(a) S_{t-1} + kh w^T and o_t = S_t^T qh, written with the decayed
    state's erased part taken out row by row."""
    c, live = s.case, s.live
    T, H, D = s.v.shape
    qh = s.q.double() / (s.q.double().pow(2).sum(2, True) + 1e-6).sqrt()
    kh = s.k.double() / (s.k.double().pow(2).sum(2, True) + 1e-6).sqrt()
    x, bias = s.raw_g.double(), s.dt_bias.double()
    if c["gate"] == "head":
        x, bias = x[:, :, None].expand(T, H, D), bias[:, None].expand(H, D)
    a = (-5.0 / (1.0 + (-(s.A_log.double().exp()[None, :, None] * (x + bias))).exp())).exp()
    if c["op"] == "kda_recurrent":
        b = 1.0 / (1.0 + (-s.raw_beta.double()).exp())
        b, w = b[:, :, None].expand(T, H, D), b[:, :, None].expand(T, H, D)
    else:
        b, w = 1.0 / (1.0 + (-s.raw_b.double()).exp()), 1.0 / (1.0 + (-s.raw_w.double()).exp())
    o = torch.zeros((T, H, D), dtype=torch.float64, device=s.v.device)
    pool = s.pool.double()
    for at in s.steps:
        seqs = torch.nonzero(at < T)[:, 0]
        t, slot = at[seqs], s.slots[:live].long()[seqs]
        S = pool[slot] * a[t][:, :, :, None]
        old = (S * (b[t] * kh[t])[:, :, :, None]).sum(2)
        S += kh[t][:, :, :, None] * (w[t] * s.v.double()[t] - old)[:, :, None, :]
        o[t] = (S * qh[t][:, :, :, None]).sum(2)
        pool[slot] = S
    return o, pool


def _exact_gated_norm(s):
    o, g, w = s.o.double(), s.gate.double(), s.weight.double()
    r = 1.0 / (o.pow(2).mean(2, True) + 1e-6).sqrt()
    sg = 1.0 / (1.0 + (-g).exp())
    silu = s.case["act"] == "silu"
    a = g * sg if silu else sg
    n = o * r
    y = n * w * a
    if not s.case["train"]:
        return y
    da = sg * (1.0 + g * (1.0 - sg)) if silu else sg * (1.0 - sg)
    dy = s.dy.double()
    dn = dy * w * a
    do = r * (dn - n * (dn * n).mean(2, True))
    return y, do, dy * n * w * da, (dy * n * a).sum((0, 1))


def _exact_block_norm(s):
    x, y, w = s.x.double(), s.y.double(), s.w_pre.double()
    kind, al = s.case["gate"], s.scale
    a = 1.0
    if kind != "none":
        a = 1.0 / (1.0 + (-s.gate.double()).exp())
        a = a if kind == "channel" else a[:, None]
    ry = 1.0 / (y.pow(2).mean(1, True) + 1e-6).sqrt()
    z = y * ry * s.w_post.double() if s.case["post"] else y
    xo = x + al * a * z
    rx = 1.0 / (xo.pow(2).mean(1, True) + 1e-6).sqrt()
    n = xo * rx
    if not s.case["train"]:
        return xo, n * w
    dh = s.dh.double()
    dn = dh * w
    dx = s.dx_out.double() + rx * (dn - n * (dn * n).mean(1, True))
    dz = al * a * dx
    got = [xo, n * w, dx]
    if s.case["post"]:
        ny = y * ry
        dny = dz * s.w_post.double()
        got += [ry * (dny - ny * (dny * ny).mean(1, True)), (dh * n).sum(0), (dz * ny).sum(0)]
    else:
        got += [dz, (dh * n).sum(0)]
    if kind != "none":
        dg = al * z * dx * a * (1.0 - a)
        got.append(dg if kind == "channel" else dg.sum(1))
    return tuple(got)


def _exact_conv(s):
    """Sequence by sequence: slices of the state's rows followed by the sequence's."""
    c, W = s.case, s.case["W"]
    x, w = s.x.double(), s.weight.double()
    b = s.bias.double() if s.bias is not None else torch.zeros(c["C"], dtype=torch.float64, device=x.device)
    train, update = c["mode"] == "train", c["mode"] == "update"
    states = s.pool.double() if update else s.init.double()
    left = states.clone()
    at = s.slots.tolist() if update else list(range(c["n"]))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db, dinit = torch.zeros_like(w), torch.zeros_like(b), torch.zeros_like(states)
    t0 = 0
    for i, m in zip(at, _lens(c)):
        xe = torch.cat([states[i], x[t0:t0 + m]])
        p = b + sum(xe[j:j + m] * w[:, j] for j in range(W))
        sg = 1.0 / (1.0 + (-p).exp())
        y[t0:t0 + m] = p * sg if c["act"] == "silu" else p
        left[i] = xe[m:]
        if train:
            dp = s.dy[t0:t0 + m].double()
            dp = dp * (sg * (1.0 + p * (1.0 - sg))) if c["act"] == "silu" else dp
            de = torch.zeros_like(xe)
            de[m:] = s.dfinal[i].double()
            for j in range(W):
                de[j:j + m] += dp * w[:, j]
                dw[:, j] += (dp * xe[j:j + m]).sum(0)
            db += dp.sum(0)
            dinit[i], dx[t0:t0 + m] = de[:W - 1], de[W - 1:]
        t0 += m
    if not train:
        return y, left
    return (y, left, dx, dw, db, dinit) if s.bias is not None else (y, left, dx, dw, dinit)
