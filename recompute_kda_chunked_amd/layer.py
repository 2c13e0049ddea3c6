"""Python binding of the operators around the chunked one: argument checks and
marshalling only, as in ``ops``. Every step runs in the HIP kernels behind
``include/kda.h``. Calls can be captured into graphs; a captured training step
takes the ``*_forward`` and ``*_backward`` functions, or autograd over leaves of
which no graph built outside the capture is alive (PyTorch's engine otherwise
ties the capture to that graph's stream).
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _DT, KdaError, _gate_flags, _raise


def _dev(t: torch.Tensor, name: str) -> torch.device:
    if t.device.type != "cuda":
        raise KdaError("inputs must be on a GPU device (%s is on %s)" % (name, t.device))
    return t.device


def _raw_stream(index):
    """The current stream's handle. torch.cuda.current_stream builds an object
    around it first, 1.9 us of a call that takes 8 in all. (Here as for the
    current device the tensors' being there means that torch.cuda is set up.)"""
    return torch._C._cuda_getCurrentRawStream(index)


def _call(dev, name, problem, *tensors, workspace=None):
    """An entry point on the current stream of the tensors' device (a launch
    goes to a stream of the current device, so another one is made current)."""
    lib = _lib.load()
    fn = getattr(lib, name)
    args = [None if t is None else t.data_ptr() for t in tensors]
    if workspace is not None:
        args += (workspace.data_ptr(), workspace.numel())
    if dev.index == torch._C._cuda_getDevice():
        st = fn(ctypes.byref(problem), *args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(ctypes.byref(problem), *args, _raw_stream(dev.index))
    if st != _lib.KDA_OK:
        _raise(lib, st, name)


def _workspace(dev, name, problem):
    nbytes = getattr(_lib.load(), name + "_workspace_bytes")(ctypes.byref(problem))
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _want(name, t, shape, dtype):
    if t is None:
        raise KdaError("%s: expected a tensor of shape %s" % (name, tuple(shape)))
    if t.shape != shape or t.dtype is not dtype:
        raise KdaError("%s: expected shape %s dtype %s, got %s %s"
                       % (name, tuple(shape), dtype, tuple(t.shape), t.dtype))


def _placed(name, t, dev, align=16):
    if t.device != dev or not t.is_contiguous() or t.data_ptr() % align:
        raise KdaError("%s must be contiguous, %d-byte aligned and on %s" % (name, align, dev))


def _rows(name, t, dev, vec):
    """The token stride (in elements, 0 for adjacent rows) of a tensor whose
    rows are contiguous; `vec`: rows start at multiples of 16 bytes."""
    if t.device != dev:
        raise KdaError("%s must be on %s" % (name, dev))
    if vec and t.data_ptr() % 16:
        raise KdaError("%s: tokens must start at multiples of 16 bytes" % name)
    if t.is_contiguous():
        return 0
    inner = t.stride()[1:]
    want, n = [], 1
    for d in reversed(t.shape[1:]):
        want.append(n)
        n *= d
    if any(a != b and d > 1 for a, b, d in zip(inner, reversed(want), t.shape[1:])):
        raise KdaError("%s: the elements of a token must be contiguous (strides %s)"
                       % (name, tuple(t.stride())))
    st = t.stride(0)
    if t.shape[0] == 1:
        return 0
    if st < n:
        raise KdaError("%s: tokens overlap (stride %d for %d elements)" % (name, st, n))
    if vec and (st * t.element_size()) % 16:
        raise KdaError("%s: tokens must start at multiples of 16 bytes" % name)
    return st


_tracing = torch._C._get_tracing_state


def _wants_grad(tensors):
    """Whether a tensor wants a gradient, or carries a forward-mode derivative
    (which no_grad does not turn off)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return forward_ad._current_level >= 0 and any(
        t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _through_autograd(*tensors):
    """Whether a call goes through its autograd function: a gradient is wanted,
    or torch.jit.trace records it (as a call of that function; the launch
    itself is no torch operation and would leave nothing in the graph)."""
    return _wants_grad(tensors) or _tracing() is not None


def _no_grad(what, instead, tensors):
    if _wants_grad(tensors):
        raise KdaError("%s is not differentiable (%s)" % (what, instead))
    if _tracing() is not None:
        raise KdaError("%s cannot be traced: its launch is no torch operation" % what)


# Tells autograd that a call has written to these tensors, so that a backward
# that kept one of them raises instead of using the new values
# (torch.autograd.graph.increment_version without its checks of types).
_overwritten = torch._C._increment_version


def _extent(t):
    """The address range a tensor's elements lie in."""
    if t.numel() == 0:
        return 0, 0
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(name, out, others):
    a0, a1 = _extent(out)
    for t in others:
        b0, b1 = _extent(t)
        if a0 < b1 and b0 < a1:
            raise KdaError("%s must not overlap an input" % name)


def _seqs(cu_seqlens, state_indices, T, slots, dev):
    """Number of sequences, with cu_seqlens and state_indices checked."""
    if cu_seqlens is None:
        N = T
    else:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.dtype is not torch.int32:
            raise KdaError("cu_seqlens: expected int32 [N+1], got %s %s"
                           % (tuple(cu_seqlens.shape), cu_seqlens.dtype))
        _placed("cu_seqlens", cu_seqlens, dev, 4)
        N = cu_seqlens.shape[0] - 1
    if state_indices is not None:
        _want("state_indices", state_indices, (N,), torch.int32)
        _placed("state_indices", state_indices, dev, 4)
        if N > 65536:
            raise KdaError("state_indices of %d sequences: not built for more than 65536" % N)
    elif slots < N:
        raise KdaError("the state pool has %d slots for %d sequences" % (slots, N))
    return N


def _new_rows(like, shape, p, cu_seqlens):
    """A decoding call's own output: rows that belong to no sequence are zero,
    written by the call itself (by a fill where no sequence launches one)."""
    if cu_seqlens is None:
        return like.new_empty(shape)
    p.zero_rest = 1
    return like.new_empty(shape) if p.n_seqs else like.new_zeros(shape)


def _recurrent(name, gates, q, k, v, raw_g, A_log, dt_bias, state, cu_seqlens, state_indices,
               scale, lower_bound, eps, gate_mode, out):
    g2 = len(gates) == 2
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise KdaError("q, k: [T,H,K]; v: [T,H,V]; state: [slots,H,K,V]")
    T, H, K = q.shape
    V, dt = v.shape[2], q.dtype
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    per_head = raw_g.dim() == 2
    gk = (T, H) if per_head else (T, H, K)
    _want("k", k, (T, H, K), dt)
    _want("v", v, (T, H, V), dt)
    _want("raw_g", raw_g, gk, dt)
    if g2:
        _want("raw_b", gates[0], (T, H, K), dt)
        _want("raw_w", gates[1], (T, H, V), dt)
    else:
        _want("raw_beta", gates[0], (T, H), dt)
    _want("A_log", A_log, (H,), torch.float32)
    _want("dt_bias", dt_bias, gk[1:], torch.float32)
    _want("state", state, (state.shape[0], H, K, V), torch.float32)
    if out is not None:
        _want("out", out, (T, H, V), dt)
    if gate_mode & _lib.KDA_GATE_PER_HEAD and not per_head:
        raise KdaError("KDA_GATE_PER_HEAD takes raw_g [T,H] and dt_bias [H]")
    if K != V or K not in (64, 128):
        raise KdaError("heads of K = %d, V = %d are not built: K = V, 64 or 128" % (K, V))
    _no_grad(name, "train with the chunked form",
             (q, k, v, raw_g, *gates, A_log, dt_bias, state, out))
    dev = _dev(q, "q")
    p = _lib.KdaRecurrentProblem(
        n_seqs=_seqs(cu_seqlens, state_indices, T, state.shape[0], dev), total_tokens=T, H=H, K=K,
        V=V, dtype=_DT[dt], gate_mode=_gate_flags(gate_mode, per_head), scale=scale,
        gate_lower_bound=lower_bound, l2_eps=eps, n_slots=state.shape[0],
        q_stride=_rows("q", q, dev, True), k_stride=_rows("k", k, dev, True),
        v_stride=_rows("v", v, dev, True), g_stride=_rows("raw_g", raw_g, dev, not per_head))
    if g2:
        p.b_stride = _rows("raw_b", gates[0], dev, True)
        p.w_stride = _rows("raw_w", gates[1], dev, True)
    else:
        p.beta_stride = _rows("raw_beta", gates[0], dev, False)
    _placed("A_log", A_log, dev)
    _placed("dt_bias", dt_bias, dev)
    _placed("state", state, dev)
    if out is None:
        out = _new_rows(q, (T, H, V), p, cu_seqlens)
    else:
        _placed("out", out, dev)
        _apart("out", out, [t for t in (q, k, v, raw_g, *gates, A_log, dt_bias, state, cu_seqlens,
                                        state_indices) if t is not None])
    _call(dev, "kda_gdn2_recurrent" if g2 else "kda_recurrent", p, q, k, v, raw_g, *gates, A_log,
          dt_bias, cu_seqlens, state_indices, state, out)
    _overwritten((state, out))
    return out


def kda_recurrent(q, k, v, raw_g, raw_beta, A_log, dt_bias, state, cu_seqlens=None, *,
                  state_indices=None, scale=1.0, lower_bound=-5.0, eps=1e-6,
                  gate_mode=_lib.KDA_GATE_SIGMOID_BOUND, out=None):
    """O [T,H,V] of the KDA operator token by token, for decoding: sequence n
    starts from its state in `state` (fp32 [slots,H,K,V]; kda_forward's final
    states serve as they are) and leaves its last state there.

    cu_seqlens: int32 [N+1] on the device, as kda_forward's (no host copy is
    needed, so the call can be captured into a graph); None: one token per
    sequence. state_indices: int32 [N] slot of each sequence (None: slot n),
    N at most 65536; a negative one marks a padded sequence, whose rows of O
    are zero and which touches no state. A slot past the pool, or one that an
    earlier sequence with tokens names too, is an error found on the device:
    NaN rows, no state touched. Rows of O that belong to no sequence are zero
    in a new O and left as they were in `out`. `state` must not overlap any
    other tensor of the call. The tokens of q, k, v, raw_g and raw_beta may be
    slices of wider rows. raw_g [T,H] with dt_bias [H] gives one gate per
    head. Not differentiable. Its time grows with the longest sequence:
    prompts belong to kda_forward."""
    return _recurrent("kda_recurrent", (raw_beta,), q, k, v, raw_g, A_log, dt_bias, state,
                      cu_seqlens, state_indices, scale, lower_bound, eps, gate_mode, out)


def gdn2_recurrent(q, k, v, raw_g, raw_b, raw_w, A_log, dt_bias, state, cu_seqlens=None, *,
                   state_indices=None, scale=1.0, lower_bound=-5.0, eps=1e-6,
                   gate_mode=_lib.KDA_GATE_SIGMOID_BOUND, out=None):
    """kda_recurrent for GDN-2: erase gate sigmoid(raw_b) [T,H,K] and write
    gate sigmoid(raw_w) [T,H,V] in place of beta (per-channel raw_g only)."""
    return _recurrent("gdn2_recurrent", (raw_b, raw_w), q, k, v, raw_g, A_log, dt_bias, state,
                      cu_seqlens, state_indices, scale, lower_bound, eps, gate_mode, out)


# ---------------------------------------------------------------------------- gated norm

_GATE_ACT = {"sigmoid": _lib.KDA_ACT_SIGMOID, "silu": _lib.KDA_ACT_SILU}


def _grad(t):
    """An output's gradient as the kernels take it: contiguous, at a multiple
    of 16 bytes."""
    if t is None:
        return None
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _gated_norm_problem(o, gate, weight, eps, activation, dy=None):
    if o.dim() < 1:
        raise KdaError("o: expected [..., V]")
    dt, V = o.dtype, o.shape[-1]
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    if activation not in _GATE_ACT:
        raise KdaError("activation must be 'sigmoid' or 'silu', got %r" % (activation,))
    _want("gate", gate, o.shape, dt)
    _want("weight", weight, (V,), torch.float32)
    if dy is not None:
        _want("dy", dy, o.shape, dt)
    if V not in (64, 128, 256):
        raise KdaError("a norm over V = %d is not built: 64, 128 or 256" % V)
    dev = _dev(o, "o")
    for name, t in (("o", o), ("gate", gate), ("weight", weight), ("dy", dy)):
        if t is not None:
            _placed(name, t, dev)
    return dev, _lib.KdaGatedNormProblem(rows=o.numel() // V, V=V, dtype=_DT[dt],
                                         activation=_GATE_ACT[activation], eps=eps)


def gated_norm_forward(o, gate, weight, *, eps=1e-6, activation="sigmoid"):
    """y = o / sqrt(mean(o^2) + eps) * weight * act(gate) over the last
    dimension (kda_gated_norm_fwd): o, gate [..., V]; weight fp32 [V]."""
    dev, p = _gated_norm_problem(o, gate, weight, eps, activation)
    y = torch.empty_like(o)
    _call(dev, "kda_gated_norm_fwd", p, o, gate, weight, y)
    return y


def gated_norm_backward(o, gate, weight, dy, *, eps=1e-6, activation="sigmoid"):
    """(do, dgate, dweight) of sum(y * dy) (kda_gated_norm_bwd), the norm
    recomputed from o; dweight fp32."""
    dev, p = _gated_norm_problem(o, gate, weight, eps, activation, dy)
    do, dgate, dw = torch.empty_like(o), torch.empty_like(gate), torch.empty_like(weight)
    _call(dev, "kda_gated_norm_bwd", p, o, gate, weight, dy, do, dgate, dw,
          workspace=_workspace(dev, "kda_gated_norm_bwd", p))
    return do, dgate, dw


class GatedNormFunction(torch.autograd.Function):
    """Autograd wrapper: saves references to the caller's inputs only."""

    @staticmethod
    def forward(ctx, o, gate, weight, eps, activation):
        ctx.save_for_backward(o, gate, weight)
        ctx.opts = dict(eps=eps, activation=activation)
        return gated_norm_forward(o, gate, weight, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return (*gated_norm_backward(*ctx.saved_tensors, _grad(dy), **ctx.opts), None, None)


def gated_norm(o, gate, weight, *, eps=1e-6, activation="sigmoid"):
    """The norm behind the operator with the output gate, differentiable:
    y = rmsnorm(o) * weight * act(gate) over each head's V channels. o and
    gate [T,H,V] (any leading dimensions), weight fp32 [V] shared by the
    heads; activation 'sigmoid' or 'silu'. V is 64, 128 or 256."""
    if _through_autograd(o, gate, weight):
        return GatedNormFunction.apply(o, gate, weight, eps, activation)
    return gated_norm_forward(o, gate, weight, eps=eps, activation=activation)


# ---------------------------------------------------------------------------- block norm


def _block_norm_problem(x, y, w_pre, w_post, raw_gate, residual_scale, eps, dx_out=None, dh=None):
    if x.dim() != 2:
        raise KdaError("x: expected [T,D], got %s" % (tuple(x.shape),))
    T, D = x.shape
    dt = x.dtype
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    _want("y", y, (T, D), dt)
    _want("w_pre", w_pre, (D,), torch.float32)
    if w_post is not None:
        _want("w_post", w_post, (D,), torch.float32)
    kind = _lib.KDA_BLOCK_GATE_NONE
    if raw_gate is not None:
        per_token = raw_gate.dim() == 1
        kind = _lib.KDA_BLOCK_GATE_TOKEN if per_token else _lib.KDA_BLOCK_GATE_CHANNEL
        _want("raw_gate", raw_gate, (T,) if per_token else (T, D), dt)
    for name, t in (("dx_out", dx_out), ("dh", dh)):
        if t is not None:
            _want(name, t, (T, D), dt)
    if not 0 < D <= 8192 or D % 8:
        raise KdaError("a norm over D = %d is not built: a multiple of 8, at most 8192" % D)
    dev = _dev(x, "x")
    for name, t in (("x", x), ("y", y), ("w_pre", w_pre), ("w_post", w_post), ("dx_out", dx_out),
                    ("dh", dh)):
        if t is not None:
            _placed(name, t, dev)
    if raw_gate is not None:
        _placed("raw_gate", raw_gate, dev,
                16 if kind == _lib.KDA_BLOCK_GATE_CHANNEL else raw_gate.element_size())
    return dev, _lib.KdaBlockNormProblem(tokens=T, D=D, dtype=_DT[dt], gate=kind,
                                         residual_scale=residual_scale, eps=eps)


def block_norm_forward(x, y, w_pre, *, w_post=None, raw_gate=None, residual_scale=1.0, eps=1e-6):
    """(x_out, h) of kda_block_norm_fwd; see block_norm."""
    dev, p = _block_norm_problem(x, y, w_pre, w_post, raw_gate, residual_scale, eps)
    x_out, h = torch.empty_like(x), torch.empty_like(x)
    _call(dev, "kda_block_norm_fwd", p, x, y, raw_gate, w_post, w_pre, x_out, h)
    return x_out, h


def block_norm_backward(x, y, w_pre, dx_out, dh, *, w_post=None, raw_gate=None,
                        residual_scale=1.0, eps=1e-6):
    """(dx, dy, dw_pre, dw_post, dgate) of sum(x_out * dx_out) + sum(h * dh)
    (kda_block_norm_bwd); either output gradient may be None (zero). dw_post
    and dgate are None without w_post and raw_gate."""
    dev, p = _block_norm_problem(x, y, w_pre, w_post, raw_gate, residual_scale, eps, dx_out, dh)
    dx, dy, dw_pre = torch.empty_like(x), torch.empty_like(y), torch.empty_like(w_pre)
    dw_post = None if w_post is None else torch.empty_like(w_post)
    dgate = None if raw_gate is None else torch.empty_like(raw_gate)
    _call(dev, "kda_block_norm_bwd", p, x, y, raw_gate, w_post, w_pre, dx_out, dh, dx, dy, dgate,
          dw_post, dw_pre, workspace=_workspace(dev, "kda_block_norm_bwd", p))
    return dx, dy, dw_pre, dw_post, dgate


class BlockNormFunction(torch.autograd.Function):
    """Autograd wrapper: saves references to the caller's inputs only."""

    @staticmethod
    def forward(ctx, x, y, w_pre, w_post, raw_gate, residual_scale, eps):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, y, w_pre, w_post, raw_gate)
        ctx.opts = dict(residual_scale=residual_scale, eps=eps)
        return block_norm_forward(x, y, w_pre, w_post=w_post, raw_gate=raw_gate, **ctx.opts)

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_out, dh):
        x, y, w_pre, w_post, raw_gate = ctx.saved_tensors
        grads = block_norm_backward(x, y, w_pre, _grad(dx_out), _grad(dh), w_post=w_post,
                                    raw_gate=raw_gate, **ctx.opts)
        return (*grads, None, None)


def block_norm(x, y, w_pre, *, w_post=None, raw_gate=None, residual_scale=1.0, eps=1e-6):
    """The step between two blocks, differentiable: the residual stream x
    [T,D] takes up the block output y [T,D], normed by w_post (fp32 [D]; None:
    as it is), times sigmoid(raw_gate) ([T] or [T,D]; None: 1) and
    residual_scale; returns (x_out, h), h = rmsnorm(x_out) * w_pre the next
    block's input. D is a multiple of 8, at most 8192."""
    if _through_autograd(x, y, w_pre, w_post, raw_gate):
        return BlockNormFunction.apply(x, y, w_pre, w_post, raw_gate, residual_scale, eps)
    return block_norm_forward(x, y, w_pre, w_post=w_post, raw_gate=raw_gate,
                              residual_scale=residual_scale, eps=eps)


# ---------------------------------------------------------------------------- short convolution

_CONV_ACT = {"silu": _lib.KDA_ACT_SILU, "none": _lib.KDA_ACT_NONE, None: _lib.KDA_ACT_NONE}


def _conv_problem(x, weight, bias, activation, **tensors):
    """(device, problem without its sequences) of a convolution over x [T,C];
    `tensors`: further arguments, name = (tensor or None, shape)."""
    if x.dim() != 2 or weight.dim() != 2:
        raise KdaError("x: expected [T,C], weight: [C,W]")
    T, C = x.shape
    dt, W = x.dtype, weight.shape[1]
    if dt not in _DT:
        raise KdaError("dtype must be float32 or bfloat16")
    if activation not in _CONV_ACT:
        raise KdaError("activation must be 'silu' or 'none', got %r" % (activation,))
    _want("weight", weight, (C, W), torch.float32)
    if bias is not None:
        _want("bias", bias, (C,), torch.float32)
    for name, (t, shape) in tensors.items():
        if t is not None:
            _want(name, t, shape, dt)
    if not 2 <= W <= 4 or C % 8 or not 0 < C <= 1 << 20:
        raise KdaError("a convolution of %d taps over %d channels is not built: 2 to 4 taps, a "
                       "multiple of 8 channels up to 2^20" % (W, C))
    dev = _dev(x, "x")
    p = _lib.KdaShortConvProblem(total_tokens=T, C=C, W=W, dtype=_DT[dt],
                                 activation=_CONV_ACT[activation],
                                 x_stride=_rows("x", x, dev, True))
    _placed("weight", weight, dev)
    if bias is not None:
        _placed("bias", bias, dev)
    for name, (t, shape) in tensors.items():
        if t is not None:
            _placed(name, t, dev)
    return dev, p


def _packed_conv_problem(x, weight, bias, cu_seqlens, activation, initial_state, dy=None,
                         d_final_state=None):
    N = 1
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.dtype is not torch.int32:
            raise KdaError("cu_seqlens: expected int32 [N+1], got %s %s"
                           % (tuple(cu_seqlens.shape), cu_seqlens.dtype))
        N = cu_seqlens.shape[0] - 1
    shape = (N, weight.shape[-1] - 1, x.shape[-1])
    dev, p = _conv_problem(x, weight, bias, activation, dy=(dy, x.shape),
                           initial_state=(initial_state, shape),
                           d_final_state=(d_final_state, shape))
    if cu_seqlens is not None:
        _placed("cu_seqlens", cu_seqlens, dev, 4)
    p.n_seqs = N
    return dev, p


def short_conv_forward(x, weight, bias=None, cu_seqlens=None, *, initial_state=None,
                       output_final_state=False, activation="silu"):
    """y, or (y, final_state), of kda_short_conv_fwd; see short_conv."""
    dev, p = _packed_conv_problem(x, weight, bias, cu_seqlens, activation, initial_state)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    final = None
    if output_final_state:
        final = torch.empty((p.n_seqs, p.W - 1, p.C), dtype=x.dtype, device=dev)
    _call(dev, "kda_short_conv_fwd", p, x, weight, bias, cu_seqlens, initial_state, y, final)
    return (y, final) if output_final_state else y


def short_conv_backward(x, weight, bias, dy, cu_seqlens=None, *, initial_state=None,
                        d_final_state=None, activation="silu"):
    """(dx, dweight, dbias, d_initial_state) of sum(y * dy) + sum(final_state
    * d_final_state) (kda_short_conv_bwd); dbias and d_initial_state are None
    without bias and initial_state."""
    dev, p = _packed_conv_problem(x, weight, bias, cu_seqlens, activation, initial_state, dy,
                                  d_final_state)
    dx, dw = torch.empty(x.shape, dtype=x.dtype, device=dev), torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dinit = None if initial_state is None else torch.empty_like(initial_state)
    _call(dev, "kda_short_conv_bwd", p, x, weight, bias, cu_seqlens, initial_state, dy,
          d_final_state, dx, dw, db, dinit, workspace=_workspace(dev, "kda_short_conv_bwd", p))
    return dx, dw, db, dinit


class ShortConvFunction(torch.autograd.Function):
    """Autograd wrapper: saves references to the caller's inputs only."""

    @staticmethod
    def forward(ctx, x, weight, bias, cu_seqlens, initial_state, final, activation):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, cu_seqlens, initial_state)
        ctx.activation = activation
        return short_conv_forward(x, weight, bias, cu_seqlens, initial_state=initial_state,
                                  output_final_state=final, activation=activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal=None):
        x, weight, bias, cu, init = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _grad(dy)
        dx, dw, db, dinit = short_conv_backward(x, weight, bias, dy, cu, initial_state=init,
                                                d_final_state=_grad(dfinal),
                                                activation=ctx.activation)
        return dx, dw, db, None, dinit, None, None


def short_conv(x, weight, bias=None, cu_seqlens=None, *, initial_state=None,
               output_final_state=False, activation="silu"):
    """The short causal convolution in front of the operator, differentiable:
    y [T,C] depthwise over the channels of x [T,C] within each packed sequence
    (cu_seqlens int32 [N+1] on the device; None: one sequence), then SiLU
    ('none': none). weight fp32 [C,W], W 2 to 4, the last tap on the token
    itself; bias fp32 [C] or None; C a multiple of 8. initial_state [N,W-1,C]
    (x's dtype): the rows before each sequence (None: zero). With
    output_final_state returns (y, final_state), final_state the last W-1 rows
    of each sequence, from which the next call or short_conv_update goes on.
    Rows of y behind the last sequence are zero."""
    if _through_autograd(x, weight, bias, initial_state):
        return ShortConvFunction.apply(x, weight, bias, cu_seqlens, initial_state,
                                       output_final_state, activation)
    return short_conv_forward(x, weight, bias, cu_seqlens, initial_state=initial_state,
                              output_final_state=output_final_state, activation=activation)


def short_conv_update(x, weight, bias, state, cu_seqlens=None, *, state_indices=None,
                      activation="silu", out=None):
    """The convolution's decoding form: y [T,C] with the rows before each
    sequence in a pool `state` [slots,W-1,C] (x's dtype; short_conv's final
    states serve as they are), which is updated in place. cu_seqlens,
    state_indices, padded sequences, rows that belong to no sequence and
    overlap as for kda_recurrent. Not differentiable."""
    if state.dim() != 3:
        raise KdaError("state: expected [slots,W-1,C], got %s" % (tuple(state.shape),))
    _no_grad("short_conv_update", "train with short_conv", (x, weight, bias, state, out))
    dev, p = _conv_problem(x, weight, bias, activation,
                           state=(state, (state.shape[0], weight.shape[-1] - 1, x.shape[-1])),
                           out=(out, x.shape))
    p.n_seqs = _seqs(cu_seqlens, state_indices, x.shape[0], state.shape[0], dev)
    p.n_slots = state.shape[0]
    if out is None:
        out = _new_rows(x, x.shape, p, cu_seqlens)
    else:
        _apart("out", out, [t for t in (x, weight, bias, state, cu_seqlens, state_indices)
                            if t is not None])
    _call(dev, "kda_short_conv_update", p, x, weight, bias, cu_seqlens, state_indices, state, out)
    _overwritten((state, out))
    return out
