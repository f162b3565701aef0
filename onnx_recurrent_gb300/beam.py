"""Thin ctypes binding of the beam search's entry points of
include/onnx_recurrent.h; argument marshalling only, as in ``ssm``.
"""
from __future__ import annotations

import ctypes
import struct
from collections import namedtuple

from . import ssm as _ssm
from .rnn import _check
from .ssm import _bad, _call, _dense, _device, _handle, _logits, _onto

_lib = None
torch = _f32 = _i32 = None

Beams = namedtuple("Beams", "parents ids scores finished")


def _load():
    global _lib, torch, _f32, _i32
    if _lib is None:
        import torch
        lib = _ssm._load()
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        lib.rnn_beam_create.argtypes = [ctypes.POINTER(vp), i64, i64]
        lib.rnn_beam_destroy.argtypes = [vp]
        lib.rnn_beam_destroy.restype = None
        lib.rnn_beam_sync.argtypes = [vp]
        lib.rnn_beam_last_launch_count.argtypes = [vp]
        lib.rnn_beam_select.argtypes = [vp, ctypes.c_char_p]
        lib.rnn_beam_reorder.argtypes = [vp, ctypes.c_char_p]
        _f32, _i32 = torch.float32, torch.int32
        _lib = lib
    return _lib


class BeamPlan:
    """A beam search plan's handle plus the attributes it was created with."""

    def __init__(self, handle, beams, end_id):
        self.handle = handle
        self.beams = beams
        self.end_id = end_id

    def __del__(self):
        try:
            if self.handle:
                rnn_beam_destroy(self)
        except Exception:
            pass


def rnn_beam_create(beams, end_id=-1) -> BeamPlan:
    """A plan for a search with ``beams`` beams an item; end_id is the token that ends a beam, -1 none."""
    h = ctypes.c_void_p()
    _check(_load().rnn_beam_create(ctypes.byref(h), int(beams), int(end_id)))
    return BeamPlan(h, int(beams), int(end_id))


def rnn_beam_destroy(plan: BeamPlan):
    if plan.handle:
        _load().rnn_beam_destroy(plan.handle)
        plan.handle = None


def rnn_beam_sync(plan: BeamPlan):
    """Wait for the device; raises if a reordering met a bad parent or slot."""
    _check(_load().rnn_beam_sync(plan.handle))


def rnn_beam_last_launch_count(plan: BeamPlan) -> int:
    return int(_load().rnn_beam_last_launch_count(plan.handle))


def _flags(t, shape, dev, name):
    """Address of a dense tensor of truth values (one byte each), 0 for None."""
    if t is None:
        return 0
    if t.dtype not in (torch.bool, torch.uint8) or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _bad(t, shape, torch.bool, dev, name)
    return t.data_ptr()


def rnn_beam_select(plan: BeamPlan, logits, scores, finished=None, parents=None, ids=None, new_scores=None,
                    new_finished=None, stream=None):
    """A step's selection into the outputs given.  logits [items * beams, vocab], or [items, vocab]: one row for all of
    an item's beams; scores [items, beams]; finished [items, beams] truth values."""
    at, stride = _logits(logits, "logits")
    dev = _device(logits, "logits")
    rows, vocab = logits.shape
    if scores.dim() != 2 or scores.shape[1] != plan.beams:
        raise ValueError(f"scores has shape {tuple(scores.shape)}, expected [items, {plan.beams}]")
    items, beams = shape = scores.shape
    shared = rows == items and beams > 1
    if not shared and rows != items * beams:
        raise ValueError(f"logits has {rows} rows, expected {items * beams} or {items}")
    args = struct.pack(
        "13q", items, vocab, _ssm._TORCH_IO[logits.dtype], at, stride, shared, _dense(scores, shape, _f32, dev, "scores"),
        _flags(finished, shape, dev, "finished"), _dense(parents, shape, _i32, dev, "parents"),
        _dense(ids, shape, _i32, dev, "ids"), _dense(new_scores, shape, _f32, dev, "new_scores"),
        _flags(new_finished, shape, dev, "new_finished"), _ssm._raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_beam_select, plan.handle, args)


def beam_select(plan: BeamPlan, logits, scores, finished=None, stream=None) -> Beams:
    """Beams(parents, ids, scores, finished), each [items, beams], best first."""
    if stream is not None:
        with _onto(stream, logits.device):
            return beam_select(plan, logits, scores, finished)
    new = lambda dtype: torch.empty(scores.shape, dtype=dtype, device=scores.device)  # noqa: E731
    r = Beams(new(_i32), new(_i32), new(_f32), new(torch.bool))
    rnn_beam_select(plan, logits, scores, finished, *r)
    return r


def rnn_beam_reorder(plan: BeamPlan, parents, tensors, outs=None, slots=None, stream=None):
    """Every beam's states become its parent's: row n * beams + b of each tensor [items * beams, ...] (or, with
    slots [items * beams], the row at that slot) that of parents[n, b].  In place without ``outs``."""
    dev = _device(parents, "parents")
    if parents.dim() != 2 or parents.shape[1] != plan.beams:
        raise ValueError(f"parents has shape {tuple(parents.shape)}, expected [items, {plan.beams}]")
    items = parents.shape[0]
    rows = items * plan.beams
    if outs is not None and len(outs) != len(tensors):
        raise ValueError(f"{len(outs)} outputs for {len(tensors)} tensors")
    fields, n_slots = [], 0
    for i, t in enumerate(tensors):
        o = t if outs is None else outs[i]
        if i == 0 and slots is not None and t.dim():
            n_slots = t.shape[0]
        count = rows if slots is None else n_slots
        if t.dim() < 1 or t.shape[0] != count:
            raise ValueError(f"a tensor has shape {tuple(t.shape)}, expected {count} rows")
        fields += (_dense(t, t.shape, t.dtype, dev, "a tensor"), _dense(o, t.shape, t.dtype, dev, "an output"),
                   t.numel() // count * t.element_size() if count else 0)
    if not fields:
        return
    table = struct.pack(f"{len(fields)}q", *fields)
    held = ctypes.create_string_buffer(table, len(table))
    args = struct.pack("7q", items, len(tensors), n_slots, _dense(parents, parents.shape, _i32, dev, "parents"),
                       _dense(slots, (rows,), _i32, dev, "slots"), ctypes.addressof(held),
                       _ssm._raw_stream(dev) if stream is None else _handle(stream))
    _call(dev, _lib.rnn_beam_reorder, plan.handle, args)


def beam_reorder(plan: BeamPlan, parents, tensors, stream=None):
    """Returns new tensors [items * beams, ...] whose rows are those of the beams' parents."""
    if stream is not None:
        with _onto(stream, parents.device):
            return beam_reorder(plan, parents, tensors)
    outs = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in tensors]
    rnn_beam_reorder(plan, parents, tensors, outs)
    return outs
