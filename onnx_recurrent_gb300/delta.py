"""Thin ctypes binding of the gated delta rule's entry points of
include/onnx_recurrent.h.

Argument marshalling only, as in ``ssm``: the ``rnn_delta_*`` functions write
into tensors the caller gives, ``delta_rule`` and ``delta_rule_grad`` allocate
their outputs.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import ssm as _ssm
from .rnn import IO_TYPES, _check
from .ssm import _call, _dense, _device, _handle, _onto, _rows, _view

_lib = None
torch = _f32 = _i32 = None


def _load():
    global _lib, torch, _f32, _i32
    if _lib is None:
        import torch
        lib = _ssm._load()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.rnn_delta_create.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i64, i32, ctypes.c_float]
        lib.rnn_delta_destroy.argtypes = [vp]
        lib.rnn_delta_destroy.restype = None
        lib.rnn_delta_set_io_type.argtypes = [vp, i32]
        lib.rnn_delta_sync.argtypes = [vp]
        lib.rnn_delta_last_launch_count.argtypes = [vp]
        lib.rnn_delta_saved_size.argtypes = [vp, i64, i64]
        lib.rnn_delta_saved_size.restype = i64
        for name in ("rule", "rule_grad", "step"):
            getattr(lib, "rnn_delta_" + name).argtypes = [vp, ctypes.c_char_p]
        _f32, _i32 = torch.float32, torch.int32
        _lib = lib
    return _lib


class Delta:
    """A gated delta rule plan's handle plus the attributes it was created with."""

    def __init__(self, handle, heads, key_heads, key_size, value_size, layout, scale):
        self.handle = handle
        self.heads = heads
        self.key_heads = key_heads
        self.key_size = key_size
        self.value_size = value_size
        self.layout = layout
        self.scale = scale
        self.io = "f32"
        self.dtype = torch.float32

    def __del__(self):
        try:
            if self.handle:
                rnn_delta_destroy(self)
        except Exception:
            pass


def rnn_delta_create(heads, key_size=128, value_size=128, key_heads=None, layout=0, scale=None) -> Delta:
    """A plan for layers of ``heads`` heads; key_heads None: one a head; scale None: 1 / sqrt(key_size)."""
    key_heads = heads if key_heads is None else key_heads
    h = ctypes.c_void_p()
    lib = _load()
    if scale is None:
        scale = 1.0 / math.sqrt(key_size) if key_size > 0 else 1.0
    _check(lib.rnn_delta_create(ctypes.byref(h), int(heads), int(key_heads), int(key_size), int(value_size), int(layout),
                                float(scale)))
    return Delta(h, int(heads), int(key_heads), int(key_size), int(value_size), int(layout), float(scale))


def rnn_delta_destroy(plan: Delta):
    if plan.handle:
        _load().rnn_delta_destroy(plan.handle)
        plan.handle = None


def rnn_delta_set_io_type(plan: Delta, io):
    """Element type of Q, K, V, Y and their gradients: "f32", "f16" or "bf16"."""
    _check(_load().rnn_delta_set_io_type(plan.handle, IO_TYPES[io] if isinstance(io, str) else int(io)))
    plan.io = io if isinstance(io, str) else {v: k for k, v in IO_TYPES.items()}[int(io)]
    plan.dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[plan.io]


def rnn_delta_sync(plan: Delta):
    """Wait for the device; raises if a call met a bad length or slot."""
    _check(_load().rnn_delta_sync(plan.handle))


def rnn_delta_last_launch_count(plan: Delta) -> int:
    return int(_load().rnn_delta_last_launch_count(plan.handle))


def rnn_delta_saved_size(plan: Delta, seq_length, batch_size) -> int:
    """Floats that rnn_delta_rule saves for rnn_delta_rule_grad."""
    return int(_load().rnn_delta_saved_size(plan.handle, int(seq_length), int(batch_size)))


def _sizes(plan, Q):
    if Q.dim() != 4:
        raise ValueError(f"Q has {Q.dim()} dimensions, expected 4")
    return (Q.shape[0], Q.shape[1]) if plan.layout == 0 else (Q.shape[1], Q.shape[0])


def _shapes(plan, S, N):
    """Shapes of Q and K, of V and Y, of g and beta, and of a state."""
    lead = (S, N) if plan.layout == 0 else (N, S)
    return (lead + (plan.key_heads, plan.key_size), lead + (plan.heads, plan.value_size), lead + (plan.heads,),
            (N, plan.heads, plan.key_size, plan.value_size))


def _inputs(plan, dev, S, N, Q, K, V, g, beta):
    qk, v, h, _ = _shapes(plan, S, N)
    io, lay = plan.dtype, plan.layout
    return (*_view(Q, qk, io, dev, "Q", lay), *_view(K, qk, io, dev, "K", lay), *_view(V, v, io, dev, "V", lay),
            *_view(g, h, _f32, dev, "g", lay), *_view(beta, h, _f32, dev, "beta", lay))


def _stream(stream, dev):
    return _ssm._raw_stream(dev) if stream is None else _handle(stream)


def rnn_delta_rule(plan: Delta, Q, K, V, g, beta, sequence_lens=None, initial_state=None, Y=None, final_state=None,
                   saved=None, stream=None):
    """The gated delta rule; Q, K [seq, batch, key_heads, key_size], V, Y [seq, batch, heads, value_size], g, beta
    [seq, batch, heads] in the plan's layout, states [batch, heads, key_size, value_size]."""
    S, N = _sizes(plan, Q)
    dev = _device(Q, "Q")
    _, v, _, st = _shapes(plan, S, N)
    args = struct.pack(
        "25q", S, N, *_inputs(plan, dev, S, N, Q, K, V, g, beta), _dense(sequence_lens, (N,), _i32, dev, "sequence_lens"),
        _dense(initial_state, st, _f32, dev, "initial_state"), *_view(Y, v, plan.dtype, dev, "Y", plan.layout),
        _dense(final_state, st, _f32, dev, "final_state"),
        0 if saved is None else _dense(saved, (rnn_delta_saved_size(plan, S, N),), _f32, dev, "saved"),
        _stream(stream, dev))
    _call(dev, _lib.rnn_delta_rule, plan.handle, args)


def delta_rule(plan: Delta, Q, K, V, g, beta, sequence_lens=None, initial_state=None, save=False, stream=None):
    """Returns (Y, final_state, saved); saved is None unless save."""
    if stream is not None:
        with _onto(stream, Q.device):
            return delta_rule(plan, Q, K, V, g, beta, sequence_lens, initial_state, save)
    S, N = _sizes(plan, Q)
    _, v, _, st = _shapes(plan, S, N)
    dev = Q.device
    Y = torch.empty(v, dtype=plan.dtype, device=dev)
    state = torch.empty(st, dtype=_f32, device=dev)
    saved = torch.empty((rnn_delta_saved_size(plan, S, N),), dtype=_f32, device=dev) if save else None
    rnn_delta_rule(plan, Q, K, V, g, beta, sequence_lens, initial_state, Y, state, saved)
    return Y, state, saved


def rnn_delta_rule_grad(plan: Delta, dY, saved, Q, K, V, g, beta, sequence_lens=None, d_final_state=None, dQ=None, dK=None,
                        dV=None, dg=None, dbeta=None, d_initial_state=None, stream=None):
    S, N = _sizes(plan, Q)
    dev, io, lay = _device(Q, "Q"), plan.dtype, plan.layout
    qk, v, h, st = _shapes(plan, S, N)
    args = struct.pack(
        "40q", S, N, *_view(dY, v, io, dev, "dY", lay), *_inputs(plan, dev, S, N, Q, K, V, g, beta),
        _dense(sequence_lens, (N,), _i32, dev, "sequence_lens"),
        _dense(saved, (rnn_delta_saved_size(plan, S, N),), _f32, dev, "saved"),
        _dense(d_final_state, st, _f32, dev, "d_final_state"), *_view(dQ, qk, io, dev, "dQ", lay),
        *_view(dK, qk, io, dev, "dK", lay), *_view(dV, v, io, dev, "dV", lay), *_view(dg, h, _f32, dev, "dg", lay),
        *_view(dbeta, h, _f32, dev, "dbeta", lay), _dense(d_initial_state, st, _f32, dev, "d_initial_state"),
        _stream(stream, dev))
    _call(dev, _lib.rnn_delta_rule_grad, plan.handle, args)


def delta_rule_grad(plan: Delta, dY, saved, Q, K, V, g, beta, sequence_lens=None, initial_state=None, d_state=None,
                    stream=None):
    """Returns a dict of dQ, dK, dV, dg, dbeta and, where initial_state is given, d_initial_state."""
    if stream is not None:
        with _onto(stream, Q.device):
            return delta_rule_grad(plan, dY, saved, Q, K, V, g, beta, sequence_lens, initial_state, d_state)
    S, N = _sizes(plan, Q)
    qk, v, h, _ = _shapes(plan, S, N)
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=Q.device)  # noqa: E731
    out = {"dQ": new(qk, plan.dtype), "dK": new(qk, plan.dtype), "dV": new(v, plan.dtype), "dg": new(h, _f32),
           "dbeta": new(h, _f32)}
    if initial_state is not None:
        out["d_initial_state"] = torch.empty_like(initial_state)
    rnn_delta_rule_grad(plan, dY, saved, Q, K, V, g, beta, sequence_lens, d_state, **out)
    return out


def rnn_delta_step(plan: Delta, Q, K, V, g, beta, state, Y, state_out=None, slots=None, stream=None):
    """One token of each row: Q, K [batch, key_heads, key_size], V, Y [batch, heads, value_size], g, beta [batch,
    heads], state [slots or batch, heads, key_size, value_size]; state_out None updates state in place."""
    dev, io = _device(Q, "Q"), plan.dtype
    N, H, dk, dv = Q.shape[0], plan.heads, plan.key_size, plan.value_size
    qk, v = (N, plan.key_heads, dk), (N, H, dv)
    n_slots = N if slots is None else state.shape[0]
    st = (n_slots, H, dk, dv)
    at = _dense(state, st, _f32, dev, "state")
    args = struct.pack(
        "24q", N, n_slots, *_rows(Q, qk, io, dev, "Q"), *_rows(K, qk, io, dev, "K"), *_rows(V, v, io, dev, "V"),
        *_rows(g, (N, H), _f32, dev, "g"), *_rows(beta, (N, H), _f32, dev, "beta"), at,
        at if state_out is None else _dense(state_out, st, _f32, dev, "state_out"), _dense(slots, (N,), _i32, dev, "slots"),
        *_rows(Y, v, io, dev, "Y"), _stream(stream, dev))
    _call(dev, _lib.rnn_delta_step, plan.handle, args)
