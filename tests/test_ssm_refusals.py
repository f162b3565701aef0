"""Refusals of the state space and token score entry points that need no GPU:
memory that an output and an input share in part.  Arguments stand in the
order of the header's structures; the addresses must not be read."""
import struct

import pytest

import onnx_recurrent_gb300 as orc


@pytest.fixture(scope="module")
def lib():
    orc.build()
    from onnx_recurrent_gb300 import ssm
    return ssm._load()


def _run(fn, fields, plan=None):
    raw = struct.pack(f"{len(fields)}q", *fields)
    return fn(plan.handle, raw) if plan else fn(raw)


def test_gradients_of_a_shared_row_need_memory_of_their_own(lib):
    at = 4096
    grad = [3, 10, -1, 0, at, 64, 64, 0, 64, 0, 0, 0, 0, at, 0, 0]
    assert _run(lib.rnn_scores_grad, grad) == 1 and "in-place" in orc.rnn_last_error()
    grad[14] = -1                                   # nor can the gradients be one row
    grad[13] = 8192
    assert _run(lib.rnn_scores_grad, grad) == 1 and "d_row_stride" in orc.rnn_last_error()
