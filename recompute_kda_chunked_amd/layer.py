"""Python binding of the operators around the chunked one: argument checks and
marshalling only, as in ``ops``. Every step runs in the HIP kernels behind
``include/kda.h``.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib
from .ops import _DT, KdaError, _gate_flags, _raise


def _dev(t: torch.Tensor, name: str) -> torch.device:
    if t.device.type != "cuda":
        raise KdaError("inputs must be on a GPU device (%s is on %s)" % (name, t.device))
    return t.device


def _on(dev: torch.device):
    """The device's context where it is not the current one (a launch goes to
    a stream of the current device)."""
    if dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _want(name, t, shape, dtype):
    if not isinstance(t, torch.Tensor):
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
    if t.is_contiguous():
        st = 0
    else:
        inner = t.stride()[1:]
        want, n = [], 1
        for d in reversed(t.shape[1:]):
            want.append(n)
            n *= d
        if any(a != b and d > 1 for a, b, d in zip(inner, reversed(want), t.shape[1:])):
            raise KdaError("%s: the elements of a token must be contiguous (strides %s)"
                           % (name, tuple(t.stride())))
        st = t.stride(0) if t.shape[0] > 1 else 0
        if t.shape[0] > 1 and st < n:
            raise KdaError("%s: tokens overlap (stride %d for %d elements)" % (name, st, n))
    if vec and (t.data_ptr() % 16 or (st * t.element_size()) % 16):
        raise KdaError("%s: tokens must start at multiples of 16 bytes" % name)
    return st


def _no_grad(what, instead, tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise KdaError("%s is not differentiable (%s)" % (what, instead))


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
    elif slots < N:
        raise KdaError("the state pool has %d slots for %d sequences" % (slots, N))
    return N


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
    _no_grad(name, "train with the chunked form", (q, k, v, raw_g, *gates, A_log, dt_bias, state))
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
        out = torch.empty((T, H, V), dtype=dt, device=dev)
    else:
        _placed("out", out, dev)
        _apart("out", out, [t for t in (q, k, v, raw_g, *gates, A_log, dt_bias, state, cu_seqlens,
                                        state_indices) if t is not None])
    lib = _lib.load()
    fn = lib.kda_gdn2_recurrent if g2 else lib.kda_recurrent
    with _on(dev):
        st = fn(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), raw_g.data_ptr(),
                *[t.data_ptr() for t in gates], A_log.data_ptr(), dt_bias.data_ptr(),
                None if cu_seqlens is None else cu_seqlens.data_ptr(),
                None if state_indices is None else state_indices.data_ptr(),
                state.data_ptr(), out.data_ptr(), _stream(dev))
    _raise(lib, st, name)
    return out


def kda_recurrent(q, k, v, raw_g, raw_beta, A_log, dt_bias, state, cu_seqlens=None, *,
                  state_indices=None, scale=1.0, lower_bound=-5.0, eps=1e-6,
                  gate_mode=_lib.KDA_GATE_SIGMOID_BOUND, out=None):
    """O [T,H,V] of the KDA operator token by token, for decoding: sequence n
    starts from its state in `state` (fp32 [slots,H,K,V]; kda_forward's final
    states serve as they are) and leaves its last state there.

    cu_seqlens: int32 [N+1] on the device, as kda_forward's (no host copy is
    needed, so the call can be captured into a graph); None: one token per
    sequence. state_indices: int32 [N] slot of each sequence (None: slot n);
    one outside [0, slots) marks a padded sequence, whose rows of O are zero
    and which touches no state. Sequences with tokens must name distinct
    slots. Rows of O behind the last sequence are not written. The tokens of
    q, k, v, raw_g and raw_beta may be slices of wider rows. raw_g [T,H] with
    dt_bias [H] gives one gate per head. Not differentiable. Its time grows
    with the longest sequence: prompts belong to kda_forward."""
    return _recurrent("kda_recurrent", (raw_beta,), q, k, v, raw_g, A_log, dt_bias, state,
                      cu_seqlens, state_indices, scale, lower_bound, eps, gate_mode, out)


def gdn2_recurrent(q, k, v, raw_g, raw_b, raw_w, A_log, dt_bias, state, cu_seqlens=None, *,
                   state_indices=None, scale=1.0, lower_bound=-5.0, eps=1e-6,
                   gate_mode=_lib.KDA_GATE_SIGMOID_BOUND, out=None):
    """kda_recurrent for GDN-2: erase gate sigmoid(raw_b) [T,H,K] and write
    gate sigmoid(raw_w) [T,H,V] in place of beta (per-channel raw_g only)."""
    return _recurrent("gdn2_recurrent", (raw_b, raw_w), q, k, v, raw_g, A_log, dt_bias, state,
                      cu_seqlens, state_indices, scale, lower_bound, eps, gate_mode, out)
