"""Thin ctypes binding of the state space and token score entry points of
include/onnx_recurrent.h.

Argument marshalling only, as in ``rnn``: the ``rnn_ssm_*`` functions write
into tensors the caller gives, the ``ssm_*`` functions and ``scores`` allocate
their outputs.  An entry point takes one structure of 8-byte fields, packed
here in one call.
"""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

from . import rnn as _rnn
from .rnn import IO_TYPES, _check

ACTIVATIONS = {None: 0, "silu": 1}
_TORCH_IO = None
_lib = None
# torch and what the calls below use of it, set by _load: a token's call takes a
# few microseconds in all, so each look-up counts.
torch = _f32 = _i32 = _empty = _empty_like = _raw_stream = _current_device = _one_device = None

Scores = namedtuple("Scores", "logp entropy lse top_ids top_logp")


def _load():
    global _lib, _TORCH_IO, torch, _f32, _i32, _empty, _empty_like, _raw_stream, _current_device, _one_device
    if _lib is None:
        import torch
        lib = _rnn.load()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.rnn_ssm_create.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i64, i32, i32, i32]
        lib.rnn_ssm_destroy.argtypes = [vp]
        lib.rnn_ssm_destroy.restype = None
        lib.rnn_ssm_set_io_type.argtypes = [vp, i32]
        lib.rnn_ssm_sync.argtypes = [vp]
        lib.rnn_ssm_last_launch_count.argtypes = [vp]
        lib.rnn_ssm_saved_size.argtypes = [vp, i64, i64]
        lib.rnn_ssm_saved_size.restype = i64
        for name in ("conv", "conv_grad", "conv_step", "scan", "scan_grad", "scan_step"):
            getattr(lib, "rnn_ssm_" + name).argtypes = [vp, ctypes.c_char_p]
        lib.rnn_scores.argtypes = [ctypes.c_char_p]
        lib.rnn_scores_grad.argtypes = [ctypes.c_char_p]
        _TORCH_IO = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
        _f32, _i32, _empty, _empty_like = torch.float32, torch.int32, torch.empty, torch.empty_like
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _one_device = torch.cuda.device_count() == 1
        _lib = lib
    return _lib


class SSM:
    """A state space plan's handle plus the attributes it was created with."""

    def __init__(self, handle, channels, state_size, groups, conv_width, layout):
        self.handle = handle
        self.channels = channels
        self.state_size = state_size
        self.groups = groups
        self.conv_width = conv_width
        self.layout = layout
        self.io = "f32"
        self.dtype = torch.float32

    def __del__(self):
        try:
            if self.handle:
                rnn_ssm_destroy(self)
        except Exception:
            pass


def rnn_ssm_create(channels, state_size=16, groups=1, conv_width=4, layout=0, activation="silu", softplus=True) -> SSM:
    """A plan for layers of ``channels`` channels; activation "silu" or None is the convolution's."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    h = ctypes.c_void_p()
    _check(_load().rnn_ssm_create(ctypes.byref(h), int(channels), int(state_size), int(groups), int(conv_width),
                                  int(layout), ACTIVATIONS[activation], int(bool(softplus))))
    return SSM(h, int(channels), int(state_size), int(groups), int(conv_width), int(layout))


def rnn_ssm_destroy(plan: SSM):
    if plan.handle:
        _load().rnn_ssm_destroy(plan.handle)
        plan.handle = None


def rnn_ssm_set_io_type(plan: SSM, io):
    """Element type of X, dt, B, C, Z, Y, the convolution's state and their gradients: "f32", "f16" or "bf16"."""
    _check(_load().rnn_ssm_set_io_type(plan.handle, IO_TYPES[io] if isinstance(io, str) else int(io)))
    plan.io = io if isinstance(io, str) else {v: k for k, v in IO_TYPES.items()}[int(io)]
    plan.dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[plan.io]


def rnn_ssm_sync(plan: SSM):
    """Wait for the device; raises if a call met a bad length or slot."""
    _check(_load().rnn_ssm_sync(plan.handle))


def rnn_ssm_last_launch_count(plan: SSM) -> int:
    return int(_load().rnn_ssm_last_launch_count(plan.handle))


def _handle(stream):
    return stream if isinstance(stream, int) else stream.cuda_stream


def _onto(stream, device):
    """`stream` as the current one: what a call allocates belongs to the stream that it runs on (memory of another
    stream's may still be in use by work queued there)."""
    if isinstance(stream, int):
        stream = torch.cuda.default_stream(device) if stream < 2 else torch.cuda.ExternalStream(stream, device)
    return torch.cuda.stream(stream)


def _call(dev, entry, handle, args):
    """An entry point, on the GPU that the call's tensors are on."""
    if _one_device or dev == _current_device():
        status = entry(handle, args)
    else:
        with torch.cuda.device(dev):
            status = entry(handle, args)
    if status:
        _check(status)


def _bad(t, shape, dtype, dev, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, strides {t.stride()}; expected {tuple(shape)}")


def _device(t, name):
    """Index of the GPU that the call's first tensor is on."""
    dev = t.get_device()            # negative for the host's
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _dense(t, shape, dtype, dev, name):
    """Address of a dense tensor of this shape and type, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _bad(t, shape, dtype, dev, name)
    return t.data_ptr()


_NO_VIEW = (0, 0, 0)


def _view(t, shape, dtype, dev, name, layout):
    """(address, step stride, row stride) of a [seq, batch, ...] (layout 0) or
    [batch, seq, ...] (layout 1) tensor whose innermost part is dense."""
    if t is None:
        return _NO_VIEW
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _bad(t, shape, dtype, dev, name)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0                  # dense
    st = t.stride()
    inner = 1
    for i in range(len(shape) - 1, 1, -1):
        if shape[i] != 1:
            if st[i] != inner:
                _bad(t, shape, dtype, dev, name + " (dense innermost part)")
            inner *= shape[i]
    ss, bs = (st[0], st[1]) if layout == 0 else (st[1], st[0])
    if ss == 0 and bs == 0:
        raise ValueError(f"{name}: steps and rows must not all share memory")
    return t.data_ptr(), ss, bs


def _rows(t, shape, dtype, dev, name):
    """The same of a [batch, ...] tensor."""
    if t is None:
        return _NO_VIEW
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _bad(t, shape, dtype, dev, name)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0
    st = t.stride()
    inner = 1
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] != 1:
            if st[i] != inner:
                _bad(t, shape, dtype, dev, name + " (dense innermost part)")
            inner *= shape[i]
    if st[0] == 0 and shape[0] > 1:
        raise ValueError(f"{name}: rows must not share memory")
    return t.data_ptr(), 0, st[0]


def _sizes(plan, X):
    if X.dim() != 3:
        raise ValueError(f"X has {X.dim()} dimensions, expected 3")
    return (X.shape[0], X.shape[1]) if plan.layout == 0 else (X.shape[1], X.shape[0])


def _shapes(plan, S, N):
    lead = (S, N) if plan.layout == 0 else (N, S)
    return lead + (plan.channels,), lead + (plan.groups, plan.state_size)


def rnn_ssm_conv(plan: SSM, X, W, bias=None, sequence_lens=None, initial_state=None, Y=None, final_state=None,
                 stream=None):
    """Y = f(causal convolution of X); every output is optional but Y."""
    S, N = _sizes(plan, X)
    D, K, dt, dev, lay = plan.channels, plan.conv_width, plan.dtype, _device(X, "X"), plan.layout
    full, _ = _shapes(plan, S, N)
    f32 = _f32
    args = struct.pack(
        "14q", S, N, *_view(X, full, dt, dev, "X", lay), _dense(W, (D, K), f32, dev, "W"),
        _dense(bias, (D,), f32, dev, "bias"), _dense(sequence_lens, (N,), _i32, dev, "sequence_lens"),
        _dense(initial_state, (N, K - 1, D), dt, dev, "initial_state"), *_view(Y, full, dt, dev, "Y", lay),
        _dense(final_state, (N, K - 1, D), dt, dev, "final_state"), _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_conv, plan.handle, args)


def ssm_conv(plan: SSM, X, W, bias=None, sequence_lens=None, initial_state=None, stream=None):
    """Returns (Y, final_state)."""
    if stream is not None:
        with _onto(stream, X.device):
            return ssm_conv(plan, X, W, bias, sequence_lens, initial_state)
    S, N = _sizes(plan, X)
    full, _ = _shapes(plan, S, N)
    Y = _empty(full, dtype=plan.dtype, device=X.device)
    state = torch.empty((N, plan.conv_width - 1, plan.channels), dtype=plan.dtype, device=X.device)
    rnn_ssm_conv(plan, X, W, bias, sequence_lens, initial_state, Y, state)
    return Y, state


def rnn_ssm_conv_grad(plan: SSM, dY, X, W, bias=None, sequence_lens=None, initial_state=None, d_final_state=None,
                      dX=None, dW=None, dbias=None, d_initial_state=None, stream=None):
    S, N = _sizes(plan, X)
    D, K, dt, dev, lay = plan.channels, plan.conv_width, plan.dtype, _device(X, "X"), plan.layout
    full, _ = _shapes(plan, S, N)
    f32, state = _f32, (N, K - 1, D)
    args = struct.pack(
        "20q", S, N, *_view(dY, full, dt, dev, "dY", lay), *_view(X, full, dt, dev, "X", lay),
        _dense(W, (D, K), f32, dev, "W"), _dense(bias, (D,), f32, dev, "bias"),
        _dense(sequence_lens, (N,), _i32, dev, "sequence_lens"),
        _dense(initial_state, state, dt, dev, "initial_state"), _dense(d_final_state, state, dt, dev, "d_final_state"),
        *_view(dX, full, dt, dev, "dX", lay), _dense(dW, (D, K), f32, dev, "dW"),
        _dense(dbias, (D,), f32, dev, "dbias"), _dense(d_initial_state, state, dt, dev, "d_initial_state"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_conv_grad, plan.handle, args)


def ssm_conv_grad(plan: SSM, dY, X, W, bias=None, sequence_lens=None, initial_state=None, d_final_state=None,
                  stream=None):
    """Returns a dict of dX and dW, of dbias where bias is given, and of d_initial_state where initial_state is."""
    if stream is not None:
        with _onto(stream, X.device):
            return ssm_conv_grad(plan, dY, X, W, bias, sequence_lens, initial_state, d_final_state)
    S, N = _sizes(plan, X)
    full, _ = _shapes(plan, S, N)
    out = {"dX": _empty(full, dtype=plan.dtype, device=X.device), "dW": torch.empty_like(W)}
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if initial_state is not None:
        out["d_initial_state"] = torch.empty_like(initial_state)
    rnn_ssm_conv_grad(plan, dY, X, W, bias, sequence_lens, initial_state, d_final_state, **out)
    return out


def rnn_ssm_conv_step(plan: SSM, X, W, bias, state, Y, state_out=None, slots=None, stream=None):
    """One token of each row: X and Y [batch, channels], state [slots or batch,
    conv_width - 1, channels]; state_out None updates state in place."""
    D, K, dt, dev = plan.channels, plan.conv_width, plan.dtype, _device(X, "X")
    N = X.shape[0]
    n_slots = N if slots is None else state.shape[0]
    shape = (n_slots, K - 1, D)
    at = _dense(state, shape, dt, dev, "state")
    args = struct.pack(
        "14q", N, n_slots, *_rows(X, (N, D), dt, dev, "X"), _dense(W, (D, K), _f32, dev, "W"),
        _dense(bias, (D,), _f32, dev, "bias"), at,
        at if state_out is None else _dense(state_out, shape, dt, dev, "state_out"),
        _dense(slots, (N,), _i32, dev, "slots"), *_rows(Y, (N, D), dt, dev, "Y"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_conv_step, plan.handle, args)


def rnn_ssm_saved_size(plan: SSM, seq_length, batch_size) -> int:
    """Floats that rnn_ssm_scan saves for rnn_ssm_scan_grad."""
    return int(_load().rnn_ssm_saved_size(plan.handle, int(seq_length), int(batch_size)))


def _scan_inputs(plan, S, N, X, dt_, A, B, C, Dskip, Z, dt_bias, lens, h0):
    D, M, io, dev, lay = plan.channels, plan.state_size, plan.dtype, X.get_device(), plan.layout
    full, bc = _shapes(plan, S, N)
    f32 = _f32
    return (*_view(X, full, io, dev, "X", lay), *_view(dt_, full, io, dev, "dt", lay),
            *_view(B, bc, io, dev, "B", lay), *_view(C, bc, io, dev, "C", lay), *_view(Z, full, io, dev, "Z", lay),
            _dense(A, (D, M), f32, dev, "A"), _dense(Dskip, (D,), f32, dev, "D"),
            _dense(dt_bias, (D,), f32, dev, "dt_bias"), _dense(lens, (N,), _i32, dev, "sequence_lens"),
            _dense(h0, (N, D, M), f32, dev, "initial_h"))


def rnn_ssm_scan(plan: SSM, X, dt, A, B, C, D=None, Z=None, dt_bias=None, sequence_lens=None, initial_h=None,
                 Y=None, Y_h=None, saved=None, stream=None):
    """The scan; X, dt, Z, Y [seq, batch, channels] and B, C [seq, batch, groups, state] in the plan's layout."""
    S, N = _sizes(plan, X)
    dev = _device(X, "X")
    full, _ = _shapes(plan, S, N)
    args = struct.pack(
        "28q", S, N, *_scan_inputs(plan, S, N, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h),
        *_view(Y, full, plan.dtype, dev, "Y", plan.layout),
        _dense(Y_h, (N, plan.channels, plan.state_size), _f32, dev, "Y_h"),
        0 if saved is None else _dense(saved, (rnn_ssm_saved_size(plan, S, N),), _f32, dev, "saved"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_scan, plan.handle, args)


def ssm_scan(plan: SSM, X, dt, A, B, C, D=None, Z=None, dt_bias=None, sequence_lens=None, initial_h=None, save=False,
             stream=None):
    """Returns (Y, Y_h, saved); saved is None unless save."""
    if stream is not None:
        with _onto(stream, X.device):
            return ssm_scan(plan, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h, save)
    S, N = _sizes(plan, X)
    full, _ = _shapes(plan, S, N)
    dev, f32 = X.device, _f32
    Y = torch.empty(full, dtype=plan.dtype, device=dev)
    Y_h = torch.empty((N, plan.channels, plan.state_size), dtype=f32, device=dev)
    saved = torch.empty((rnn_ssm_saved_size(plan, S, N),), dtype=f32, device=dev) if save else None
    rnn_ssm_scan(plan, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h, Y, Y_h, saved)
    return Y, Y_h, saved


def rnn_ssm_scan_grad(plan: SSM, dY, saved, X, dt, A, B, C, D=None, Z=None, dt_bias=None, sequence_lens=None,
                      initial_h=None, dY_h=None, dX=None, ddt=None, dB=None, dC=None, dZ=None, dA=None, dD=None,
                      ddt_bias=None, d_initial_h=None, stream=None):
    S, N = _sizes(plan, X)
    io, dev, lay, f32 = plan.dtype, _device(X, "X"), plan.layout, _f32
    full, bc = _shapes(plan, S, N)
    ch, st = (plan.channels,), (N, plan.channels, plan.state_size)
    args = struct.pack(
        "47q", S, N, *_view(dY, full, io, dev, "dY", lay),
        *_scan_inputs(plan, S, N, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h),
        _dense(saved, (rnn_ssm_saved_size(plan, S, N),), f32, dev, "saved"), _dense(dY_h, st, f32, dev, "dY_h"),
        *_view(dX, full, io, dev, "dX", lay), *_view(ddt, full, io, dev, "ddt", lay),
        *_view(dB, bc, io, dev, "dB", lay), *_view(dC, bc, io, dev, "dC", lay), *_view(dZ, full, io, dev, "dZ", lay),
        _dense(dA, ch + (plan.state_size,), f32, dev, "dA"), _dense(dD, ch, f32, dev, "dD"),
        _dense(ddt_bias, ch, f32, dev, "ddt_bias"), _dense(d_initial_h, st, f32, dev, "d_initial_h"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_scan_grad, plan.handle, args)


def ssm_scan_grad(plan: SSM, dY, saved, X, dt, A, B, C, D=None, Z=None, dt_bias=None, sequence_lens=None,
                  initial_h=None, dY_h=None, stream=None):
    """Returns a dict of dX, ddt, dA, dB, dC and of dD, dZ, ddt_bias, d_initial_h for those of the inputs given."""
    if stream is not None:
        with _onto(stream, X.device):
            return ssm_scan_grad(plan, dY, saved, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h, dY_h)
    S, N = _sizes(plan, X)
    full, bc = _shapes(plan, S, N)
    new = lambda shape: torch.empty(shape, dtype=plan.dtype, device=X.device)  # noqa: E731
    out = {"dX": new(full), "ddt": new(full), "dB": new(bc), "dC": new(bc), "dA": torch.empty_like(A)}
    if Z is not None:
        out["dZ"] = new(full)
    if D is not None:
        out["dD"] = torch.empty_like(D)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty_like(dt_bias)
    if initial_h is not None:
        out["d_initial_h"] = torch.empty_like(initial_h)
    rnn_ssm_scan_grad(plan, dY, saved, X, dt, A, B, C, D, Z, dt_bias, sequence_lens, initial_h, dY_h, **out)
    return out


def rnn_ssm_scan_step(plan: SSM, X, dt, A, B, C, H, Y, D=None, Z=None, dt_bias=None, H_out=None, slots=None,
                      stream=None):
    """One token of each row: X, dt, Z, Y [batch, channels], B, C [batch, groups,
    state], H [slots or batch, channels, state]; H_out None updates H in place."""
    dev, io, f32 = _device(X, "X"), plan.dtype, _f32
    N, ch, M = X.shape[0], plan.channels, plan.state_size
    full, bc = (N, ch), (N, plan.groups, M)
    n_slots = N if slots is None else H.shape[0]
    at = _dense(H, (n_slots, ch, M), f32, dev, "H")
    args = struct.pack(
        "27q", N, n_slots, *_rows(X, full, io, dev, "X"), *_rows(dt, full, io, dev, "dt"),
        *_rows(B, bc, io, dev, "B"), *_rows(C, bc, io, dev, "C"),
        *_rows(Z, full, io, dev, "Z"), _dense(A, (ch, M), f32, dev, "A"), _dense(D, (ch,), f32, dev, "D"),
        _dense(dt_bias, (ch,), f32, dev, "dt_bias"), at,
        at if H_out is None else _dense(H_out, (n_slots, ch, M), f32, dev, "H_out"),
        _dense(slots, (N,), _i32, dev, "slots"), *_rows(Y, full, io, dev, "Y"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_ssm_scan_step, plan.handle, args)


_SHARED_ROW = -1        # RNN_SHARED_ROW: every row is the same one
_LSE_PAIR = 256         # RNN_SCORES_LSE_PAIR: lse is [2, rows]


def _untouched(t):
    """Whether no torch operation has written to an lse of ``_new_lse``."""
    try:
        return t._version == 1
    except RuntimeError:                    # made in inference mode, which does not count
        return True


def _new_lse(rows, device):
    """An lse of [rows] with room behind it for what its rounding leaves off."""
    t = _empty(2 * rows, dtype=_f32, device=device).resize_(rows)
    t._rest = True
    return t


def _lse(t, rows, dev):
    """(address, flag of io) of an lse: [rows], or [2, rows] with its rounding's rest, which ``_new_lse``'s have too."""
    if t is None:
        return 0, 0
    if t.dim() == 2:
        return _dense(t, (2, rows), _f32, dev, "lse"), _LSE_PAIR
    return _dense(t, (rows,), _f32, dev, "lse"), _LSE_PAIR if getattr(t, "_rest", False) and _untouched(t) else 0


def _logits(t, name, dtype=None, shape=None, device=None):
    """(address, row stride) of a [rows, vocab] tensor with dense rows; rows
    that are all one row (an expanded tensor's) have no stride of their own."""
    if not t.is_cuda or (device is not None and t.device != device):
        raise TypeError(f"{name} must be a CUDA tensor on one device with the others")
    if t.dim() != 2 or (shape is not None and t.shape != shape) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype or 'rows of logits'} {tuple(shape or ())}")
    if t.dtype not in _TORCH_IO:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    rows, vocab = t.shape
    if t.is_contiguous():
        return t.data_ptr(), vocab
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a row must be dense")
    return t.data_ptr(), (t.stride(0) or _SHARED_ROW) if rows > 1 else vocab


def _scores(_, args):
    return _lib.rnn_scores(args)


def _scores_grad(_, args):
    return _lib.rnn_scores_grad(args)


def rnn_scores(logits, ids=None, top=0, logp=None, entropy=None, lse=None, top_ids=None, top_logp=None, stream=None):
    """Scores of rows of logits [rows, vocab] into the outputs given; an lse of [2, rows] takes its rounding's rest too."""
    _load()
    at, stride = _logits(logits, "logits")
    rows, vocab = logits.shape
    dev, f32, i32, top = logits.get_device(), _f32, _i32, int(top)
    lse, pair = _lse(lse, rows, dev)
    args = struct.pack(
        "13q", rows, vocab, stride, _TORCH_IO[logits.dtype] + pair, at, _dense(ids, (rows,), i32, dev, "ids"), top,
        _dense(logp, (rows,), f32, dev, "logp"), _dense(entropy, (rows,), f32, dev, "entropy"), lse,
        _dense(top_ids, (rows, top), i32, dev, "top_ids"), _dense(top_logp, (rows, top), f32, dev, "top_logp"),
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _scores, None, args)


def scores(logits, ids=None, top=0, stream=None) -> Scores:
    """Scores(logp, entropy, lse, top_ids, top_logp) of rows of logits; logp is
    None without ids, top_ids and top_logp are None for top = 0."""
    _load()
    if stream is not None:
        with _onto(stream, logits.device):
            return scores(logits, ids, top)
    at, stride = _logits(logits, "logits")
    device, rows, top = logits.device, logits.shape[0], int(top)
    if top < 0:
        raise ValueError(f"top must not be negative, got {top}")
    dev, entropy = logits.get_device(), _empty(rows, dtype=_f32, device=device)
    top_logp = _empty((rows, top), dtype=_f32, device=device) if top else None
    r = Scores(None if ids is None else _empty_like(entropy), entropy, _new_lse(rows, device),
               _empty_like(top_logp, dtype=_i32) if top else None, top_logp)
    ids_at = _dense(ids, (rows,), _i32, dev, "ids")
    args = struct.pack(
        "13q", rows, logits.shape[1], stride, _TORCH_IO[logits.dtype] + _LSE_PAIR, at, ids_at, top,
        r.logp.data_ptr() if ids_at else 0, entropy.data_ptr(), r.lse.data_ptr(), r.top_ids.data_ptr() if top else 0,
        top_logp.data_ptr() if top else 0, _raw_stream(dev))
    _call(dev, _scores, None, args)
    return r


def rnn_scores_grad(logits, ids, result: Scores, d_logp=None, d_entropy=None, d_top=None, dlogits=None, stream=None):
    """Gradient of the scores in the logits into dlogits (which may be logits of rows of their own); ``result`` is
    their Scores."""
    _load()
    at, stride = _logits(logits, "logits")
    rows, vocab = logits.shape
    d_at, d_stride = _logits(dlogits, "dlogits", logits.dtype, logits.shape, logits.device)
    if d_stride == _SHARED_ROW:
        raise ValueError("dlogits: rows must not share memory")
    dev, f32 = logits.get_device(), _f32
    top = 0 if d_top is None else d_top.shape[1]
    lse, pair = _lse(result.lse, rows, dev)
    args = struct.pack(
        "16q", rows, vocab, stride, _TORCH_IO[logits.dtype] + pair, at, _dense(ids, (rows,), _i32, dev, "ids"),
        lse, _dense(result.entropy, (rows,), f32, dev, "entropy"),
        _dense(d_logp, (rows,), f32, dev, "d_logp"), _dense(d_entropy, (rows,), f32, dev, "d_entropy"), top,
        _dense(result.top_ids, (rows, top), _i32, dev, "top_ids") if top else 0,
        _dense(d_top, (rows, top), f32, dev, "d_top"), d_at, d_stride,
        _raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _scores_grad, None, args)


def scores_grad(logits, ids, result: Scores, d_logp=None, d_entropy=None, d_top=None, stream=None):
    """Returns dlogits, in the logits' type."""
    _load()
    if stream is not None:
        with _onto(stream, logits.device):
            return scores_grad(logits, ids, result, d_logp, d_entropy, d_top)
    dlogits = _empty(logits.shape, dtype=logits.dtype, device=logits.device)
    rnn_scores_grad(logits, ids, result, d_logp, d_entropy, d_top, dlogits)
    return dlogits
