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


def test_outputs_whose_steps_or_rows_share_memory(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3, groups=2)
    S, N, D, at = 5, 2, 8, 4096
    bad = [(0, 64), (64, 0), (4, 64), (64, 4), (16, 16)]         # step and row strides
    dense = (at, 0, 0)
    for ss, bs in bad:
        out = (at, ss, bs)
        conv = [S, N, *dense, at, 0, 0, 0, *out, 0, 0]
        conv_grad = [S, N, *dense, *dense, at, 0, 0, 0, 0, *out, 0, 0, 0, 0]
        scan = [S, N, *dense, *dense, *dense, *dense, 0, 0, 0, at, 0, 0, 0, 0, *out, 0, 0, 0]
        assert (len(conv), len(conv_grad), len(scan)) == (14, 20, 28)
        for name, fields in (("conv", conv), ("conv_grad", conv_grad), ("scan", scan)):
            assert _run(getattr(lib, "rnn_ssm_" + name), fields, p) == 1, (name, ss, bs)
            assert "share memory" in orc.rnn_last_error()
        for which in range(5):                       # dX, ddt, dB, dC, dZ
            outs = [0] * 15
            outs[3 * which:3 * which + 3] = out
            fields = [S, N] + [*dense] * 6 + [at, 0, 0, 0, 0, at, 0] + outs + [0] * 5
            assert len(fields) == 47 and _run(lib.rnn_ssm_scan_grad, fields, p) == 1, which
            assert "share memory" in orc.rnn_last_error()
    row = (at, 0, 4)
    step = [N, 0, *dense, at, 0, at, at, 0, *row, 0]
    assert _run(lib.rnn_ssm_conv_step, step, p) == 1 and "share memory" in orc.rnn_last_error()
    step = [N, 0] + [*dense] * 4 + [0, 0, 0, at, 0, 0, at, at, 0, *row, 0]
    assert len(step) == 27 and _run(lib.rnn_ssm_scan_step, step, p) == 1 and "share memory" in orc.rnn_last_error()


def test_outputs_that_do_not_share_memory_pass_the_check(lib):
    """Strides of a part of a wider tensor, either dimension first; a stride of a dimension of one value is not read.
    (The next refusal shows that the check was passed.)"""
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    for S, N, ss, bs in ((5, 2, 16, 8), (5, 2, 8, 40), (1, 2, 0, 8), (5, 1, 8, 0), (1, 1, 3, 3)):
        conv = [S, N, 4096, 0, 0, 4096, 0, 0, 0, 4096, ss, bs, 2, 0]        # final_state not aligned
        assert _run(lib.rnn_ssm_conv, conv, p) == 1 and "final_state" in orc.rnn_last_error()


def test_states_that_overlap_in_part(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    at, h, bytes_ = 4096, 1 << 20, 2 * 8 * 4 * 4
    for other in (h + 4, h - 4, h + bytes_ - 4, h - bytes_ + 4):
        scan = [5, 2] + [at, 0, 0] * 4 + [0, 0, 0, at, 0, 0, 0, h, at, 0, 0, other, 0, 0]
        assert _run(lib.rnn_ssm_scan, scan, p) == 1 and "overlap" in orc.rnn_last_error()


def test_slopes_of_the_scans_states_that_overlap_in_part(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    at, h, bytes_ = 4096, 1 << 20, 2 * 8 * 4 * 4
    for other in (h + 4, h - 4, h + bytes_ - 4, h - bytes_ + 4):
        grad = [5, 2] + [at, 0, 0] * 6 + [at, 0, 0, 0, 0, at, h] + [0] * 15 + [0, 0, 0, other, 0]
        assert len(grad) == 47 and _run(lib.rnn_ssm_scan_grad, grad, p) == 1 and "overlap" in orc.rnn_last_error()


def test_slopes_of_the_convolutions_states_that_overlap_in_part(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    at, h, bytes_ = 4096, 1 << 20, 2 * 2 * 8 * 4
    for other in (h + 4, h - 4, h + bytes_ - 4, h - bytes_ + 4):
        grad = [5, 2, at, 0, 0, at, 0, 0, at, 0, 0, 0, h, 0, 0, 0, 0, 0, other, 0]
        assert len(grad) == 20 and _run(lib.rnn_ssm_conv_grad, grad, p) == 1 and "overlap" in orc.rnn_last_error()


def test_the_convolutions_and_single_tokens_states_that_overlap_in_part(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    at, h = 4096, 1 << 20
    for slots, n in ((0, 2), (at, 7)):
        for step, size in (("conv", 2 * 8 * 4), ("scan", 8 * 4 * 4)):
            for other in (h + 4, h - 4, h + n * size - 4, h - n * size + 4):
                if step == "conv":
                    fields = [2, n, at, 0, 0, at, 0, h, other, slots, at, 0, 0, 0]
                else:
                    fields = [2, n] + [at, 0, 0] * 4 + [0, 0, 0, at, 0, 0, h, other, slots, at, 0, 0, 0]
                assert _run(getattr(lib, f"rnn_ssm_{step}_step"), fields, p) == 1, (step, other)
                assert "overlap" in orc.rnn_last_error()
    for other in (h + 4, h - 4, h + 124, h - 124):
        conv = [5, 2, at, 0, 0, at, 0, 0, h, at, 0, 0, other, 0]
        assert _run(lib.rnn_ssm_conv, conv, p) == 1 and "overlap" in orc.rnn_last_error()


def test_the_convolution_in_place(lib):
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    x, y, w = (1 << 20, 0, 0), (2 << 20, 0, 0), 4096
    assert _run(lib.rnn_ssm_conv, [50, 2, *x, w, 0, 0, 0, *x, 0, 0], p) == 1 and "Y must not be X" in orc.rnn_last_error()
    for dX in (x, y):
        assert _run(lib.rnn_ssm_conv_grad, [50, 2, *y, *x, w, 0, 0, 0, 0, *dX, 0, 0, 0, 0], p) == 1
        assert "dX must not be" in orc.rnn_last_error()
