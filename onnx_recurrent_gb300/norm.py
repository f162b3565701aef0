"""Thin ctypes binding of the layer normalisation's entry points of
include/onnx_recurrent.h; argument marshalling only, as in ``ssm``.
"""
from __future__ import annotations

import ctypes
import struct

from . import ssm as _ssm
from .rnn import IO_TYPES, _check
from .ssm import _SHARED_ROW, _bad, _call, _dense, _device, _handle, _onto

_lib = None
torch = _f32 = None


def _load():
    global _lib, torch, _f32
    if _lib is None:
        import torch
        lib = _ssm._load()
        vp = ctypes.c_void_p
        lib.rnn_norm_create.argtypes = [ctypes.POINTER(vp), ctypes.c_int64, ctypes.c_float]
        lib.rnn_norm_destroy.argtypes = [vp]
        lib.rnn_norm_destroy.restype = None
        lib.rnn_norm_set_io_type.argtypes = [vp, ctypes.c_int]
        lib.rnn_norm_last_launch_count.argtypes = [vp]
        lib.rnn_layer_norm.argtypes = [vp, ctypes.c_char_p]
        lib.rnn_layer_norm_grad.argtypes = [vp, ctypes.c_char_p]
        _f32 = torch.float32
        _lib = lib
    return _lib


class Norm:
    """A normalisation plan's handle plus the attributes it was created with."""

    def __init__(self, handle, size, eps):
        self.handle = handle
        self.size = size
        self.eps = eps
        self.io = "f32"
        self.dtype = torch.float32

    def __del__(self):
        try:
            if self.handle:
                rnn_norm_destroy(self)
        except Exception:
            pass


def rnn_norm_create(size, eps=1e-5) -> Norm:
    """A plan for rows of ``size`` values."""
    h = ctypes.c_void_p()
    _check(_load().rnn_norm_create(ctypes.byref(h), int(size), float(eps)))
    return Norm(h, int(size), float(eps))


def rnn_norm_destroy(plan: Norm):
    if plan.handle:
        _load().rnn_norm_destroy(plan.handle)
        plan.handle = None


def rnn_norm_set_io_type(plan: Norm, io):
    """Element type of X, Y and their gradients: "f32", "f16" or "bf16"."""
    _check(_load().rnn_norm_set_io_type(plan.handle, IO_TYPES[io] if isinstance(io, str) else int(io)))
    plan.io = io if isinstance(io, str) else {v: k for k, v in IO_TYPES.items()}[int(io)]
    plan.dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[plan.io]


def rnn_norm_last_launch_count(plan: Norm) -> int:
    return int(_load().rnn_norm_last_launch_count(plan.handle))


def _rows(plan, t, name, shape, dev, out=False):
    """(address, row stride) of a [..., size] tensor whose rows are dense and evenly apart; an input's may all be one."""
    if t is None:
        return 0, 0
    if t.dtype is not plan.dtype or t.get_device() != dev or t.shape != shape:
        _bad(t, shape, plan.dtype, dev, name)
    if t.is_contiguous():
        return t.data_ptr(), 0
    size, st = t.shape, t.stride()
    if size[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name}: a row must be dense")
    stride, count = None, 1
    for i in range(len(size) - 2, -1, -1):
        if size[i] == 1:
            continue
        if stride is None:
            stride = st[i]
        elif st[i] != stride * count:
            raise ValueError(f"{name}: rows must be evenly apart")
        count *= size[i]
    if stride == 0:
        if out:
            raise ValueError(f"{name}: rows must not share memory")
        stride = _SHARED_ROW
    return t.data_ptr(), stride or 0


def _count(plan, X):
    if X.dim() < 1 or X.shape[-1] != plan.size:
        raise ValueError(f"X has shape {tuple(X.shape)}, expected rows of {plan.size}")
    return X.numel() // plan.size


def rnn_layer_norm(plan: Norm, X, W=None, bias=None, Y=None, stats=None, stream=None):
    """Y = (X - mean) rstd W + bias over the last dimension; stats [rows, 2] takes mean and rstd.  Y may be X."""
    dev = _device(X, "X")
    rows, d, shape = _count(plan, X), (plan.size,), X.shape
    args = struct.pack(
        "9q", rows, *_rows(plan, X, "X", shape, dev), _dense(W, d, _f32, dev, "W"), _dense(bias, d, _f32, dev, "bias"),
        *_rows(plan, Y, "Y", shape, dev, True), _dense(stats, (rows, 2), _f32, dev, "stats"),
        _ssm._raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_layer_norm, plan.handle, args)


def layer_norm(plan: Norm, X, W=None, bias=None, stream=None):
    """Returns (Y, stats)."""
    if stream is not None:
        with _onto(stream, X.device):
            return layer_norm(plan, X, W, bias)
    Y = torch.empty_like(X, memory_format=torch.contiguous_format)      # (of the plan's type, or the call refuses X)
    stats = torch.empty((_count(plan, X), 2), dtype=_f32, device=X.device)
    rnn_layer_norm(plan, X, W, bias, Y, stats)
    return Y, stats


def rnn_layer_norm_grad(plan: Norm, dY, X, stats, W=None, dX=None, dW=None, dbias=None, stream=None):
    dev = _device(X, "X")
    rows, d = _count(plan, X), (plan.size,)
    args = struct.pack(
        "12q", rows, *_rows(plan, dY, "dY", X.shape, dev), *_rows(plan, X, "X", X.shape, dev),
        _dense(stats, (rows, 2), _f32, dev, "stats"), _dense(W, d, _f32, dev, "W"), *_rows(plan, dX, "dX", X.shape, dev, True),
        _dense(dW, d, _f32, dev, "dW"), _dense(dbias, d, _f32, dev, "dbias"),
        _ssm._raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_layer_norm_grad, plan.handle, args)


def layer_norm_grad(plan: Norm, dY, X, stats, W=None, bias=None, stream=None):
    """Returns a dict of dX and of dW and dbias for those of W and bias given."""
    if stream is not None:
        with _onto(stream, X.device):
            return layer_norm_grad(plan, dY, X, stats, W, bias)
    out = {"dX": torch.empty_like(X, memory_format=torch.contiguous_format)}
    if W is not None:
        out["dW"] = torch.empty_like(W)
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    rnn_layer_norm_grad(plan, dY, X, stats, W, **out)
    return out
