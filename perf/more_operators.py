"""Cases for measuring the operators of a state-space layer: the selective scan over packed
sequences (prompts and training), its decoding form on a pool of states, and the group norm behind
it with its activation or gate.

``own`` selects the framework's kernels; otherwise ``run`` computes the same with elementary
torch operations in fp32 (the scan in chunks, gradients by torch's autograd). ``exact`` computes
it in fp64 from the definitions, with hand-written gradients.
"""
from __future__ import annotations

import math
import random

import torch

own = False

F32, BF16 = "float32", "bfloat16"
INF = float("inf")


# ---------------------------------------------------------------------------- cases


def listed():
    return [
        # one short prompt through a small fp32 model's layer: latency alone counts
        _scan("scan_prompt_37x8x64x64_f32", F32, T=37, n=1, H=8, G=1, N=64, P=64),
        # a packed batch of prompts, some continued from earlier states, B and C shared by all heads
        _scan("scan_prompt_4099x48x128x64_bf16", BF16, T=4099, n=9, H=48, G=1, N=128, P=64,
              init=True, fused=True),
        # one long prompt at few heads: parallel along the sequence or not at all
        _scan("scan_prompt_32771x16x64x128_bf16", BF16, T=32771, n=1, H=16, G=2, N=64, P=128),
        # a small ragged fp32 training batch with states and limits on the step size
        _scan("scan_1531x12x64x64_f32_train", F32, T=1531, n=6, H=12, G=2, N=64, P=64, init=True,
              limit=True, train=True),
        # a training step at 8K tokens x 64 heads, packed documents
        _scan("scan_8192x64x128x64_bf16_train", BF16, T=8192, n=3, H=64, G=8, N=128, P=64,
              fused=True, train=True),
        # one user's decoding step at the small model's sizes: latency again
        _rec("step_1x8x64x64_f32", F32, n=1, H=8, G=1, N=64, P=64, L=1),
        # a large decoding batch padded to a fixed launch size, states scattered over a pool
        _rec("step_193x64x128x64_bf16", BF16, n=193, H=64, G=8, N=128, P=64, L=1, pad=3),
        # ragged runs of up to 6 drafted tokens a sequence, some sequences with none
        _rec("draft_33x48x128x64_bf16", BF16, n=33, H=48, G=1, N=128, P=64, L=6),
        # the norm behind the scan of a decoding batch: gate first, not centred
        _norm("group_norm_16x4096_bf16", BF16, T=16, groups=8, W=512, gate="first", center=False),
        # the same in a training step at 8K tokens
        _norm("group_norm_8192x4096_bf16_train", BF16, T=8192, groups=8, W=512, gate="first",
              center=False, train=True),
        # one group per head, centred, with bias and the gate behind; odd sizes, fp32
        _norm("group_norm_1021x2400_f32_train", F32, T=1021, groups=12, W=200, gate="after",
              center=True, bias=True, train=True),
        # centred groups with an activation and no gate
        _norm("group_norm_4097x2560_bf16", BF16, T=4097, groups=40, W=64, gate="none", center=True,
              bias=True),
    ]


def _scan(name, dtype, T, n, H, G, N, P, init=False, limit=False, fused=False, train=False):
    c = {"op": "ssm_scan", "dtype": dtype, "T": T, "n": n, "H": H, "G": G, "N": N, "P": P,
         "init": init, "limit": limit, "fused": fused, "train": train}
    return dict(c, name=name) if name else c


def _rec(name, dtype, n, H, G, N, P, L, pad=0, fused=True):
    c = {"op": "ssm_recurrent", "dtype": dtype, "n": n, "H": H, "G": G, "N": N, "P": P, "L": L,
         "pad": pad, "fused": fused, "limit": False}
    return dict(c, name=name) if name else c


def _norm(name, dtype, T, groups, W, gate, center, act="silu", bias=False, train=False):
    c = {"op": "group_norm", "dtype": dtype, "T": T, "groups": groups, "W": W, "gate": gate,
         "center": center, "act": act, "bias": bias, "train": train}
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ssm_scan", "ssm_scan", "ssm_recurrent", "group_norm"])
    dtype = rng.choice([F32, BF16, BF16])
    if op == "group_norm":
        W = 8 * _spread(rng, 1, 512)
        groups = _spread(rng, 1, max(1, 8192 // W))
        T = _spread(rng, 1, min(16384, (1 << 24) // (W * groups)))
        gate = rng.choice(["none", "after", "first"])
        return _norm(None, dtype, T, groups, W, gate, rng.random() < 0.5,
                     rng.choice(["silu", "silu", "sigmoid"]), rng.random() < 0.5,
                     rng.random() < 0.6)
    N, P, G = rng.choice([64, 128]), rng.choice([64, 128]), rng.choice([1, 1, 2, 8])
    H = G * _spread(rng, 1, 64 // G)
    if op == "ssm_recurrent":
        L = rng.choice([1, 1, _spread(rng, 2, 12)])
        room = 193 * 64 * 128 * 64 // (H * N * P * max(1, L // 3))
        n = _spread(rng, 1, max(1, min(256, room)))
        return _rec(None, dtype, n, H, G, N, P, L, rng.choice([0, 0, rng.randint(1, 4)]),
                    rng.random() < 0.5)
    most = 8192 * 64 * 128 * 64 // (1 if dtype == BF16 else 4)
    T = _spread(rng, 1, min(32768, most // (H * N * P)))
    return _scan(None, dtype, T, _spread(rng, 1, min(T, 40)), H, G, N, P, rng.random() < 0.5,
                 rng.random() < 0.3, rng.random() < 0.5, T <= 8192 and rng.random() < 0.6)


def _lens(case):
    """Tokens of each sequence, the same for every seed: of a decoding case (up to L each, the
    first one L, some of them none), of a scan (T tokens cut at random places)."""
    r = random.Random("%s %s" % (case["n"], case.get("L", case.get("T"))))
    if "L" in case:
        return [case["L"]] + [case["L"] if case["L"] == 1 else r.randint(0, case["L"])
                              for _ in range(case["n"] - 1)]
    cuts = sorted(r.randint(0, case["T"]) for _ in range(case["n"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "group_norm":
        n, gated = case["T"] * case["groups"] * case["W"], case["gate"] != "none"
        if case["train"]:  # x, gate, dy in; y, dx, dgate out
            return {"bytes": (6 if gated else 4) * n * e, "flops": 40 * n}
        return {"bytes": (3 if gated else 2) * n * e, "flops": 15 * n}
    H, G, N, P = case["H"], case["G"], case["N"], case["P"]
    states = case["n"] * H * N * P * 4
    if case["op"] == "ssm_recurrent":
        rows = sum(_lens(case))
        return {"bytes": 2 * states + rows * (2 * H * P + 2 * G * N + H) * e,
                "flops": rows * H * 5 * N * P}
    T, train = case["T"], case["train"]
    row = 2 * H * P + 2 * G * N + H  # x, y, B, C and the step sizes
    ends = states * (1 + case["init"])
    if train:  # dy; dx, dB, dC and the step sizes' gradient
        row += 2 * H * P + 2 * G * N + H
        ends *= 2
    return {"bytes": T * row * e + ends, "flops": T * H * N * P * (12 if train else 4)}


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

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    if case["op"] == "group_norm":
        T, C = case["T"], case["groups"] * case["W"]
        s.x = randn(T, C, scale=0.7, shift=0.1)
        s.gate = None if case["gate"] == "none" else randn(T, C)
        s.weight = randn(C, dtype=torch.float32, scale=0.2, shift=1.0)
        s.bias = randn(C, dtype=torch.float32, scale=0.2) if case["bias"] else None
        s.dy = randn(T, C) if case["train"] else None
        s.leaves = tuple(t for t in (s.x, s.weight, s.bias, s.gate) if t is not None)
    else:
        _prepare_ssm(s, case, gen, randn, rand)
    if case.get("train"):
        for t in s.leaves:
            t.requires_grad_(True)
    return s


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _prepare_ssm(s, case, gen, randn, rand):
    n, H, G, N, P = (case[k] for k in ("n", "H", "G", "N", "P"))
    lens = _lens(case)
    rows = sum(lens)
    T = rows + case.get("pad", 0) if case.get("L") == 1 else rows  # a padded sequence has one token, or none
    if case["fused"]:  # slices of the convolution's output, as the layer hands them on
        xbc = randn(T, H * P + 2 * G * N, scale=0.7)
        x, b, c = xbc.split([H * P, G * N, G * N], dim=1)
        s.x, s.B, s.C = x.view(T, H, P), b.view(T, G, N), c.view(T, G, N)
    else:
        s.x, s.B, s.C = (randn(T, H, P, scale=0.7), randn(T, G, N, scale=0.7),
                         randn(T, G, N, scale=0.7))
    s.raw_dt = randn(T, H)
    s.A_log = torch.log(1.0 + 15.0 * rand(H))
    s.D = randn(H, dtype=torch.float32, scale=0.1, shift=1.0)
    # step sizes around 0.001 to 0.1: the bias is their softplus' inverse
    first = torch.exp(math.log(1e-3) + math.log(100.0) * rand(H))
    s.dt_bias = first + torch.log(-torch.expm1(-first))
    s.limit = (0.004, 0.12) if case["limit"] else (0.0, INF)
    s.cu = _cu(lens + [0] * (case.get("pad", 0) if case.get("L", 1) > 1 else 0))
    if case["op"] == "ssm_recurrent":
        slots, pad = n + n // 4 + 1, case["pad"]
        s.pool = randn(slots, H, N, P, dtype=torch.float32, scale=0.3)
        s.slots = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
        if pad:  # a batch filled up to its launch size: no state behind the last ones
            s.slots = torch.cat([s.slots, torch.full((pad,), -1, dtype=torch.int32, device="cuda")])
        if case["L"] == 1:
            s.cu = None
        s.live = n
        # row of the j-th token of each sequence; T (a row of padding) where it has none
        at = [sum(lens[:i]) for i in range(n)]
        s.steps = torch.tensor([[at[i] + j if j < lens[i] else T for i in range(n)]
                                for j in range(case["L"])], device="cuda")
        return
    s.init = randn(n, H, N, P, dtype=torch.float32, scale=0.3) if case["init"] else None
    s.dy, s.dfinal = None, None
    if case["train"]:
        s.dy, s.dfinal = randn(T, H, P), randn(n, H, N, P, dtype=torch.float32, scale=0.3)
    s.leaves = tuple(t for t in (s.x, s.raw_dt, s.A_log, s.B, s.C, s.D, s.dt_bias, s.init)
                     if t is not None)
    if case["train"] and case["fused"]:  # leaves that are slices
        s.x, s.B, s.C = (t.detach() for t in (s.x, s.B, s.C))
        s.leaves = (s.x, s.raw_dt, s.A_log, s.B, s.C, *s.leaves[5:])
    _plain_chunks(s, lens)


CHUNK = 64  # of the plain form


def _plain_chunks(s, lens):
    """The plain form's chunks: by position in their sequence, the sequences with more chunks
    first, so that those still running at a position are the first few of it."""
    order = sorted(range(len(lens)), key=lambda i: -(-(-lens[i] // CHUNK)))
    start = [sum(lens[:i]) for i in range(len(lens))]
    T, rows, s.active = sum(lens), [], []
    while True:
        k = len(s.active)
        live = [i for i in order if lens[i] > k * CHUNK]
        if not live:
            break
        s.active.append(len(live))
        rows += [[start[i] + k * CHUNK + j if k * CHUNK + j < lens[i] else T for j in range(CHUNK)]
                 for i in live]
    s.rows = torch.tensor(rows, device="cuda").reshape(-1, CHUNK)
    at = torch.empty(T, dtype=torch.long)
    flat = s.rows.reshape(-1).cpu()
    real = flat < T
    at[flat[real]] = torch.nonzero(real)[:, 0]
    s.back = at.cuda()  # where each token lies among the chunks' rows
    s.order = torch.tensor(order, device="cuda")
    s.unorder = torch.argsort(s.order)


# ---------------------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    c = s.case
    if c["op"] == "ssm_recurrent":
        return _plain_recurrent(s)
    if c["op"] == "group_norm":
        y = _plain_group_norm(s)
        if not c["train"]:
            return y
        return (y.detach(), *torch.autograd.grad(y, s.leaves, s.dy))
    y, final = _plain_scan(s)
    if not c["train"]:
        return y, final
    return (y.detach(), final.detach(), *torch.autograd.grad((y, final), s.leaves, (s.dy, s.dfinal)))


def _run_own(s):
    import recompute_kda_chunked_amd as kda
    c = s.case
    if c["op"] == "ssm_recurrent":
        y = kda.ssm_recurrent(s.x, s.raw_dt, s.A_log, s.B, s.C, s.D, s.dt_bias, s.pool, s.cu,
                              state_indices=s.slots, dt_limit=s.limit)
        return y, s.pool
    if c["op"] == "group_norm":
        y = kda.group_norm(s.x, s.weight, s.bias, s.gate, groups=c["groups"], center=c["center"],
                           gate_first=c["gate"] == "first", activation=c["act"])
        if not c["train"]:
            return y
        return (y.detach(), *torch.autograd.grad(y, s.leaves, s.dy))
    y, final = kda.ssm_scan(s.x, s.raw_dt, s.A_log, s.B, s.C, s.D, s.dt_bias, s.cu,
                            initial_state=s.init, output_final_state=True, dt_limit=s.limit)
    if not c["train"]:
        return y, final
    return (y.detach(), final.detach(), *torch.autograd.grad((y, final), s.leaves, (s.dy, s.dfinal)))


# ---------------------------------------------------------------------------- plain forms


def _softplus(z):
    return torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-torch.abs(z)))


def _plain_dt(s):
    return torch.clamp(_softplus(s.raw_dt.float() + s.dt_bias), s.limit[0], s.limit[1])


def _heads(t, H):
    """[..., G, N] -> [..., H, N]: the heads of a group share its rows."""
    return t.repeat_interleave(H // t.shape[-2], dim=-2)


def _plain_scan(s):
    c = s.case
    H, G, N, P = (c[k] for k in ("H", "G", "N", "P"))

    def chunks(t):  # [T, h, d] -> [chunks, h, CHUNK, d], zeros where a chunk has no token
        t = torch.cat([t, t.new_zeros((1, *t.shape[1:]))])
        return t[s.rows].transpose(1, 2)

    x, B, C = (chunks(t.float()) for t in (s.x, s.B, s.C))
    dt = chunks(_plain_dt(s)[..., None])[..., 0]  # [chunks, H, CHUNK]
    cum = torch.cumsum(-torch.exp(s.A_log)[:, None] * dt, -1)
    total = cum[..., -1:]
    later = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=x.device).triu(1)
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(later, -INF))
    pairs = torch.matmul(C, B.transpose(2, 3)).repeat_interleave(H // G, dim=1)
    y = torch.matmul(pairs * decay * dt[..., None, :], x)
    Bh, Ch = (t.repeat_interleave(H // G, dim=1) for t in (B, C))
    local = torch.matmul((Bh * (torch.exp(total - cum) * dt)[..., None]).transpose(2, 3), x)
    state = x.new_zeros((c["n"], H, N, P)) if s.init is None else s.init
    state = state[s.order]
    enter, left, at = [], [], 0
    for i, m in enumerate(s.active):
        left.append(state[m:])
        state = state[:m]
        enter.append(state)
        state = state * torch.exp(total[at:at + m])[..., None] + local[at:at + m]
        at += m
    left.append(state)
    final = torch.cat(left[::-1])[s.unorder]
    y = y + torch.matmul(Ch * torch.exp(cum)[..., None], torch.cat(enter))
    y = y.transpose(1, 2).reshape(-1, H, P)[s.back] + s.D[:, None] * s.x.float()
    return y.to(s.dtype), final


def _plain_recurrent(s):
    c = s.case
    H = c["H"]
    x, B, C, dt = s.x.float(), _heads(s.B.float(), H), _heads(s.C.float(), H), _plain_dt(s)
    decay = torch.exp(-torch.exp(s.A_log) * dt)
    state = s.pool.index_select(0, s.slots[:s.live])
    out = torch.zeros((x.shape[0] + 1, *x.shape[1:]), dtype=s.dtype, device=x.device)

    def padded(t, value=0.0):
        return torch.cat([t, t.new_full((1, *t.shape[1:]), value)])

    x, B, C, dt, decay = padded(x), padded(B), padded(C), padded(dt), padded(decay, 1.0)
    for at in s.steps:
        xt = x[at]
        state = state * decay[at][..., None, None] + (dt[at][..., None] * B[at])[..., None] * xt[..., None, :]
        y = torch.matmul(C[at][..., None, :], state)[..., 0, :] + s.D[:, None] * xt
        out[at] = y.to(s.dtype)
    s.pool.index_copy_(0, s.slots[:s.live].long(), state)
    return out[:-1], s.pool


def _plain_group_norm(s):
    c = s.case
    shape = (c["T"], c["groups"], c["W"])
    x = s.x.float()
    act = None
    if s.gate is not None:
        g = s.gate.float()
        act = torch.sigmoid(g)
        act = g * act if c["act"] == "silu" else act
        x = x * act if c["gate"] == "first" else x
    x = x.reshape(shape)
    if c["center"]:
        x = x - x.mean(-1, keepdim=True)
    n = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).reshape(s.x.shape)
    y = n * s.weight
    y = y if s.bias is None else y + s.bias
    if c["gate"] == "none":
        a = torch.sigmoid(y)
        y = y * a if c["act"] == "silu" else a
    elif c["gate"] == "after":
        y = y * act
    return y.to(s.dtype)


# ---------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "ssm_recurrent":
            return _exact_recurrent(s)
        if case["op"] == "group_norm":
            return _exact_group_norm(s)
        if max(_lens(case)) > 12000:
            return _exact_scan_by_tokens(s)
        return _exact_scan(s)


def _exact_dt(s):
    z = s.raw_dt.double() + s.dt_bias.double()
    dt = torch.where(z > 0, z + (1.0 + (-z.abs()).exp()).log(), (1.0 + (-z.abs()).exp()).log())
    # log(1 + e) of a small e, from its series
    e = (-z.abs()).exp()
    small = e < 1e-5
    series = e - e * e / 2 + e * e * e / 3
    dt = torch.where(small, torch.where(z > 0, z + series, series), dt)
    inside = (dt > s.limit[0]) & (dt < s.limit[1])
    return dt.clamp(*s.limit), inside, 1.0 / (1.0 + (-z).exp())


def _exact_recurrent(s):
    c = s.case
    T, H, P = s.x.shape
    per = H // c["G"]
    dt, A = _exact_dt(s)[0], s.A_log.double().exp()
    y = torch.zeros((T, H, P), dtype=torch.float64, device=s.x.device)
    pool = s.pool.double()
    for at in s.steps:
        seqs = torch.nonzero(at < T)[:, 0]
        t, slot = at[seqs], s.slots[:s.live].long()[seqs]
        for h in range(H):
            x, b, q = s.x[t, h].double(), s.B[t, h // per].double(), s.C[t, h // per].double()
            S = pool[slot, h] * (-A[h] * dt[t, h]).exp()[:, None, None]
            S = S + (dt[t, h][:, None] * b)[:, :, None] * x[:, None, :]
            y[t, h] = (S * q[:, :, None]).sum(1) + s.D[h].double() * x
            pool[slot, h] = S
    return y, pool


def _exact_scan_by_tokens(s):
    """A long sequence without gradients: token by token, every head at once."""
    c = s.case
    per = c["H"] // c["G"]
    dt, A = _exact_dt(s)[0], s.A_log.double().exp()
    y = torch.empty(s.x.shape, dtype=torch.float64, device=s.x.device)
    final = torch.zeros((c["n"], c["H"], c["N"], c["P"]), dtype=torch.float64, device=s.x.device)
    if s.init is not None:
        final += s.init.double()
    if c["train"] or c["T"] > 65536:
        return None
    decay, xd = (-A * dt).exp(), s.x.double() * dt[..., None]
    b, q = (t.double().repeat_interleave(per, 1) for t in (s.B, s.C))
    t = 0
    for n, m in enumerate(_lens(c)):
        S = final[n]
        for t in range(t, t + m):
            S.mul_(decay[t][:, None, None]).baddbmm_(b[t][:, :, None], xd[t][:, None, :])
            torch.bmm(q[t][:, None, :], S, out=y[t][:, None, :])
        t = t + 1 if m else t
    return y + s.D.double()[:, None] * s.x.double(), final


def _exact_scan(s):
    """Sequence by sequence and head by head with every pair of tokens:
    y = (L o C B^T) (dt x) + e^cum C S0 + D x, and its gradients by the product rule."""
    c = s.case
    T, H, P = s.x.shape
    N, per, train = c["N"], H // c["G"], c["train"]
    dt, inside, slope = _exact_dt(s)
    A, D, dev = s.A_log.double().exp(), s.D.double(), s.x.device

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device=dev)

    y, final = zeros(T, H, P), zeros(c["n"], H, N, P)
    dx, dB, dC, ddt, dl = zeros(T, H, P), zeros(T, c["G"], N), zeros(T, c["G"], N), zeros(T, H), zeros(T, H)
    dinit = zeros(c["n"], H, N, P)
    t0 = 0
    for n, m in enumerate(_lens(c)):
        r = slice(t0, t0 + m)
        t0 += m
        for h in range(H):
            S0 = s.init[n, h].double() if s.init is not None else zeros(N, P)
            dST = s.dfinal[n, h].double() if train else None
            if m == 0:
                final[n, h] = S0
                if train:
                    dinit[n, h] = dST
                continue
            x, b, q, d = s.x[r, h].double(), s.B[r, h // per].double(), s.C[r, h // per].double(), dt[r, h]
            cum = torch.cumsum(-A[h] * d, 0)
            L = (cum[:, None] - cum[None, :]).tril_().exp_().tril_()
            LG = L * (q @ b.t())
            e, rest, tot = cum.exp()[:, None], (cum[-1] - cum).exp()[:, None], cum[-1].exp()
            xd = d[:, None] * x
            y[r, h] = LG @ xd + e * (q @ S0) + D[h] * x
            final[n, h] = (rest * b).t() @ xd + tot * S0
            if not train:
                continue
            dy = s.dy[r, h].double()
            bS, Sdy = b @ dST, dy @ S0.t()
            dxd = LG.t() @ dy + rest * bS
            dx[r, h] = d[:, None] * dxd + D[h] * dy
            ddt[r, h] = (x * dxd).sum(1)
            pair = dy @ xd.t()
            F = LG.mul_(pair)
            pair.mul_(L)
            dC[r, h // per] += pair @ b + e * Sdy
            dB[r, h // per] += pair.t() @ q + rest * (xd @ dST.t())
            out = rest[:, 0] * (xd * bS).sum(1)
            dcum = F.sum(1) - F.sum(0) + e[:, 0] * (q * Sdy).sum(1) - out
            dcum[-1] += out.sum() + tot * (S0 * dST).sum()
            dl[r, h] = dcum.flip(0).cumsum(0).flip(0)
            dinit[n, h] = tot * dST + (e * q).t() @ dy
    if not train:
        return y, final
    draw_dt = (ddt - A * dl) * slope * inside
    got = [y, final, dx, draw_dt, (-A * dt * dl).sum(0), dB, dC, (s.x.double() * s.dy.double()).sum((0, 2)),
           draw_dt.sum(0)]
    return tuple(got + ([dinit] if s.init is not None else []))


def _exact_group_norm(s):
    c = s.case
    T, C = s.x.shape
    groups = (T, c["groups"], c["W"])
    x, w = s.x.double(), s.weight.double()
    b = s.bias.double() if s.bias is not None else torch.zeros_like(w)
    silu, kind = c["act"] == "silu", c["gate"]

    def act(v):
        sg = 1.0 / (1.0 + (-v).exp())
        return (v * sg, sg * (1.0 + v / (1.0 + v.exp()))) if silu else (sg, sg / (1.0 + v.exp()))

    def mean(v):
        return v.reshape(groups).mean(2, True).expand(groups).reshape(T, C)

    a, da = act(s.gate.double()) if kind != "none" else (None, None)
    z = x * a if kind == "first" else x
    z = z - mean(z) if c["center"] else z
    r = 1.0 / (mean(z * z) + 1e-6).sqrt()
    n = z * r
    p = n * w + b
    if kind == "none":
        y, slope = act(p)
    else:
        y, slope = (p * a, a) if kind == "after" else (p, 1.0)
    if not c["train"]:
        return y
    dy = s.dy.double()
    dp = dy * slope
    dn = dp * w
    dz = r * (dn - n * mean(dn * n) - (mean(dn) if c["center"] else 0.0))
    got = [y, dz * a if kind == "first" else dz, (dp * n).sum(0)]
    if s.bias is not None:
        got.append(dp.sum(0))
    if kind != "none":
        got.append(dz * x * da if kind == "first" else dy * p * da)
    return tuple(got)
