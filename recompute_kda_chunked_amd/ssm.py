"""Python binding of a state-space layer's operators: the selective scan, its
decoding form and the group norm behind it. Argument checks and marshalling
only, as in ``layer``; every step runs in the HIP kernels behind
``include/kda.h``.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .layer import (_apart, _call, _dev, _grad, _new_rows, _no_grad, _overwritten, _placed, _rows,
                    _seqs, _through_autograd, _want, _workspace)
from .ops import _DT, KdaError

_INF = float("inf")


def _ssm_problem(x, raw_dt, A_log, B, C, D, dt_bias, dt_limit):
    """(device, problem without its sequences) of a scan over x [T,H,P]."""
    if x.dim() != 3 or B.dim() != 3:
        raise KdaError("x: expected [T,H,P], B and C: [T,G,N]")
    T, H, P = x.shape
    G, N = B.shape[1:]
    dt = x.dtype
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    _want("raw_dt", raw_dt, (T, H), dt)
    _want("A_log", A_log, (H,), torch.float32)
    _want("B", B, (T, G, N), dt)
    _want("C", C, (T, G, N), dt)
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _want(name, t, (H,), torch.float32)
    if H < 1 or G < 1 or H % G:
        raise KdaError("%d heads in %d groups: the groups must divide the heads" % (H, G))
    if N not in (64, 128) or P not in (64, 128):
        raise KdaError("states of N = %d, P = %d are not built: 64 or 128 each" % (N, P))
    lo, hi = dt_limit
    if not 0 <= lo <= hi or lo == _INF:
        raise KdaError("dt_limit: expected 0 <= lower <= upper, got %r" % (dt_limit,))
    dev = _dev(x, "x")
    p = _lib.KdaSsmProblem(total_tokens=T, H=H, G=G, N=N, P=P, dtype=_DT[dt], dt_min=lo, dt_max=hi,
                           x_stride=_rows("x", x, dev, True),
                           dt_stride=_rows("raw_dt", raw_dt, dev, False),
                           B_stride=_rows("B", B, dev, True), C_stride=_rows("C", C, dev, True))
    for name, t in (("A_log", A_log), ("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _placed(name, t, dev)
    return dev, p


def _scan_problem(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, dt_limit, **tensors):
    """(device, problem) of a packed scan; `tensors`: further arguments, name =
    (tensor or None, True for a state, False for rows like x's)."""
    dev, p = _ssm_problem(x, raw_dt, A_log, B, C, D, dt_bias, dt_limit)
    p.n_seqs = 1
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.dtype is not torch.int32:
            raise KdaError("cu_seqlens: expected int32 [N+1], got %s %s"
                           % (tuple(cu_seqlens.shape), cu_seqlens.dtype))
        _placed("cu_seqlens", cu_seqlens, dev, 4)
        p.n_seqs = cu_seqlens.shape[0] - 1
    for name, (t, is_state) in tensors.items():
        if t is not None:
            if is_state:
                _want(name, t, (p.n_seqs, p.H, p.N, p.P), torch.float32)
            else:
                _want(name, t, x.shape, x.dtype)
            _placed(name, t, dev)
    return dev, p


def ssm_scan_forward(x, raw_dt, A_log, B, C, D=None, dt_bias=None, cu_seqlens=None, *,
                     initial_state=None, output_final_state=False, dt_limit=(0.0, _INF)):
    """y, or (y, final_state), of kda_ssm_fwd; see ssm_scan."""
    dev, p = _scan_problem(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, dt_limit,
                           initial_state=(initial_state, True))
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    final = None
    if output_final_state:
        final = torch.empty((p.n_seqs, p.H, p.N, p.P), dtype=torch.float32, device=dev)
    _call(dev, "kda_ssm_fwd", p, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state, y,
          final, workspace=_workspace(dev, "kda_ssm_fwd", p))
    return (y, final) if output_final_state else y


def ssm_scan_backward(x, raw_dt, A_log, B, C, D, dt_bias, dy, cu_seqlens=None, *,
                      initial_state=None, d_final_state=None, dt_limit=(0.0, _INF)):
    """(dx, draw_dt, dA_log, dB, dC, dD, ddt_bias, d_initial_state) of
    sum(y * dy) + sum(final_state * d_final_state) (kda_ssm_bwd), everything
    else recomputed from the inputs; dD, ddt_bias and d_initial_state are None
    without D, dt_bias and initial_state."""
    dev, p = _scan_problem(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, dt_limit, dy=(dy, False),
                           initial_state=(initial_state, True), d_final_state=(d_final_state, True))
    dx, ddt, dB, dC = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (x, raw_dt, B, C))
    dA = torch.empty_like(A_log)
    dD, dbias, dinit = (None if t is None else torch.empty_like(t) for t in (D, dt_bias, initial_state))
    _call(dev, "kda_ssm_bwd", p, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state, dy,
          d_final_state, dx, ddt, dA, dB, dC, dD, dbias, dinit,
          workspace=_workspace(dev, "kda_ssm_bwd", p))
    return dx, ddt, dA, dB, dC, dD, dbias, dinit


class SsmScanFunction(torch.autograd.Function):
    """Autograd wrapper: saves references to the caller's inputs only."""

    @staticmethod
    def forward(ctx, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state, final, dt_limit):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state)
        ctx.dt_limit = dt_limit
        return ssm_scan_forward(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens,
                                initial_state=initial_state, output_final_state=final,
                                dt_limit=dt_limit)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal=None):
        x, raw_dt, A_log, B, C, D, dt_bias, cu, init = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _grad(dy)
        *grads, dinit = ssm_scan_backward(x, raw_dt, A_log, B, C, D, dt_bias, dy, cu,
                                          initial_state=init, d_final_state=_grad(dfinal),
                                          dt_limit=ctx.dt_limit)
        return (*grads, None, dinit, None, None)


def ssm_scan(x, raw_dt, A_log, B, C, D=None, dt_bias=None, cu_seqlens=None, *, initial_state=None,
             output_final_state=False, dt_limit=(0.0, _INF)):
    """The selective scan of a state-space layer over packed sequences, for
    prompts and training, differentiable: y [T,H,P] with, per sequence and
    head h, of group h // (H // G),
      dt = clamp(softplus(raw_dt + dt_bias), *dt_limit)
      S = exp(-exp(A_log) dt) S + dt B x^T,  y = S^T C + D x.
    x [T,H,P], raw_dt [T,H], B and C [T,G,N] may have tokens that are slices
    of wider rows, as short_conv's output has them; A_log, D and dt_bias fp32
    [H], the last two None for zero; N and P 64 or 128; cu_seqlens int32 [n+1]
    on the device (None: one sequence; no host copy is needed, so the call can
    be captured into a graph). initial_state fp32 [n,H,N,P] (None: zero). With
    output_final_state returns (y, final_state), from which the next call or
    ssm_recurrent goes on. Rows of y that belong to no sequence are zero. No
    gradient reaches raw_dt where a limit holds. NaN and infinities reach y and
    the final state only where the formulas have them; of the gradients they may
    reach others of their chunk (128 tokens from the sequence's first, 64 for
    fp32). The workspace is the states'
    size every 128 tokens (64 for fp32) and for each sequence, of x's type
    forward, fp32 and twice backward; up to as much again where long sequences
    are divided."""
    if _through_autograd(x, raw_dt, A_log, B, C, D, dt_bias, initial_state):
        return SsmScanFunction.apply(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens, initial_state,
                                     output_final_state, dt_limit)
    return ssm_scan_forward(x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens,
                            initial_state=initial_state, output_final_state=output_final_state,
                            dt_limit=dt_limit)


def ssm_recurrent(x, raw_dt, A_log, B, C, D, dt_bias, state, cu_seqlens=None, *,
                  state_indices=None, dt_limit=(0.0, _INF), out=None):
    """The selective scan token by token, for decoding: y [T,H,P], sequence n
    starting from its state in `state` (fp32 [slots,H,N,P]; ssm_scan's final
    states serve as they are) and leaving its last state there. Per head h, of group h // (H // G), with dt =
    clamp(softplus(raw_dt + dt_bias), *dt_limit):
    S = exp(-exp(A_log) dt) S + dt B x^T, y = S^T C + D x. x [T,H,P], raw_dt
    [T,H], B and C [T,G,N] may have tokens that are slices of wider rows;
    A_log, D and dt_bias fp32 [H], the last two None for zero; N and P 64 or
    128. cu_seqlens, state_indices, padded sequences, rows that belong to no
    sequence and overlap as for kda_recurrent. Not differentiable."""
    if state.dim() != 4:
        raise KdaError("state: expected [slots,H,N,P], got %s" % (tuple(state.shape),))
    _no_grad("ssm_recurrent", "train with ssm_scan", (x, raw_dt, A_log, B, C, D, dt_bias, state, out))
    dev, p = _ssm_problem(x, raw_dt, A_log, B, C, D, dt_bias, dt_limit)
    _want("state", state, (state.shape[0], p.H, p.N, p.P), torch.float32)
    _placed("state", state, dev)
    p.n_seqs = _seqs(cu_seqlens, state_indices, p.total_tokens, state.shape[0], dev)
    p.n_slots = state.shape[0]
    if out is None:
        out = _new_rows(x, x.shape, p, cu_seqlens)
    else:
        _want("out", out, x.shape, x.dtype)
        _placed("out", out, dev)
        _apart("out", out, [t for t in (x, raw_dt, A_log, B, C, D, dt_bias, state, cu_seqlens,
                                        state_indices) if t is not None])
    _call(dev, "kda_ssm_recurrent", p, x, raw_dt, A_log, B, C, D, dt_bias, cu_seqlens,
          state_indices, state, out)
    _overwritten((state, out))
    return out


# ---------------------------------------------------------------------------- group norm

_ACT = {"silu": _lib.KDA_ACT_SILU, "sigmoid": _lib.KDA_ACT_SIGMOID, "none": _lib.KDA_ACT_NONE,
        None: _lib.KDA_ACT_NONE}


def _group_norm_problem(x, weight, bias, gate, groups, eps, activation, center, gate_first, dy=None):
    if x.dim() < 1:
        raise KdaError("x: expected [..., C]")
    C, dt = x.shape[-1], x.dtype
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    if activation not in _ACT:
        raise KdaError("activation must be 'silu', 'sigmoid' or 'none', got %r" % (activation,))
    if gate is None and gate_first:
        raise KdaError("gate_first takes a gate")
    if gate is not None and _ACT[activation] == _lib.KDA_ACT_NONE:
        raise KdaError("a gate takes the activation 'silu' or 'sigmoid'")
    _want("weight", weight, (C,), torch.float32)
    if bias is not None:
        _want("bias", bias, (C,), torch.float32)
    for name, t in (("gate", gate), ("dy", dy)):
        if t is not None:
            _want(name, t, x.shape, dt)
    if not isinstance(groups, int) or groups < 1 or C < 1 or C % groups:
        raise KdaError("groups = %r must divide the %d channels" % (groups, C))
    if (C // groups) % 8 or C // groups > 8192 or C > 1 << 20:
        raise KdaError("groups of %d of %d channels are not built: multiples of 8 up to 8192, 2^20 "
                       "channels in all" % (C // groups, C))
    dev = _dev(x, "x")
    kind = (_lib.KDA_GROUP_GATE_NONE if gate is None else
            _lib.KDA_GROUP_GATE_FIRST if gate_first else _lib.KDA_GROUP_GATE_AFTER)
    p = _lib.KdaGroupNormProblem(rows=x.numel() // C, C=C, groups=groups, dtype=_DT[dt], gate=kind,
                                 activation=_ACT[activation], center=bool(center), eps=eps)
    if x.dim() == 2:  # a row may be a slice of a wider one
        p.x_stride = _rows("x", x, dev, True)
        p.gate_stride = 0 if gate is None else _rows("gate", gate, dev, True)
    for name, t in (("x", x), ("gate", gate)) if x.dim() != 2 else ():
        if t is not None:
            _placed(name, t, dev)
    for name, t in (("weight", weight), ("bias", bias), ("dy", dy)):
        if t is not None:
            _placed(name, t, dev)
    return dev, p


def group_norm_forward(x, weight, bias=None, gate=None, *, groups, eps=1e-6, activation="silu",
                       center=True, gate_first=False):
    """y of kda_group_norm_fwd; see group_norm."""
    dev, p = _group_norm_problem(x, weight, bias, gate, groups, eps, activation, center, gate_first)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _call(dev, "kda_group_norm_fwd", p, x, gate, weight, bias, y)
    return y


def group_norm_backward(x, weight, bias, gate, dy, *, groups, eps=1e-6, activation="silu",
                        center=True, gate_first=False):
    """(dx, dweight, dbias, dgate) of sum(y * dy) (kda_group_norm_bwd), the
    norm recomputed from x and gate; dbias and dgate are None without bias and
    gate."""
    dev, p = _group_norm_problem(x, weight, bias, gate, groups, eps, activation, center, gate_first,
                                 dy)
    dx, dw = torch.empty(x.shape, dtype=x.dtype, device=dev), torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dgate = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    _call(dev, "kda_group_norm_bwd", p, x, gate, weight, bias, dy, dx, dgate, dw, db,
          workspace=_workspace(dev, "kda_group_norm_bwd", p))
    return dx, dw, db, dgate


class GroupNormFunction(torch.autograd.Function):
    """Autograd wrapper: saves references to the caller's inputs only."""

    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, eps, activation, center, gate_first):
        ctx.save_for_backward(x, weight, bias, gate)
        ctx.opts = dict(groups=groups, eps=eps, activation=activation, center=center,
                        gate_first=gate_first)
        return group_norm_forward(x, weight, bias, gate, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return (*group_norm_backward(*ctx.saved_tensors, _grad(dy), **ctx.opts), *(None,) * 5)


def group_norm(x, weight, bias=None, gate=None, *, groups, eps=1e-6, activation="silu",
               center=True, gate_first=False):
    """Group norm over the channels of each token (channels last), with an
    activation or an activated gate, differentiable. x [..., C] in `groups`
    groups of adjacent channels, weight and bias (None: zero) fp32 [C]:
    n = (z - mean) / sqrt(var + eps) per token and group (center=False: the
    mean stays, var is the mean square), p = n * weight + bias, and
      no gate:           z = x,              y = act(p)
      gate:              z = x,              y = p * act(gate)
      gate, gate_first:  z = x * act(gate),  y = p
    act is 'silu' or 'sigmoid', without a gate also 'none'. x and gate [T,C]
    may have rows that are slices of wider ones. C / groups is a multiple of 8
    up to 8192."""
    if _through_autograd(x, weight, bias, gate):
        return GroupNormFunction.apply(x, weight, bias, gate, groups, eps, activation, center,
                                       gate_first)
    return group_norm_forward(x, weight, bias, gate, groups=groups, eps=eps, activation=activation,
                              center=center, gate_first=gate_first)
