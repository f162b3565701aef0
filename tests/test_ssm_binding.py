"""The binding's choice of device, without a GPU: stand-ins for the library and its tensors."""
import contextlib
import struct

import pytest
import torch

import onnx_recurrent_gb300 as orc
from onnx_recurrent_gb300 import ssm


class FakeTensor:
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.device = torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        st = torch.empty(self.shape, device="meta").stride()
        return st if i is None else st[i]

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """(current device, entry point, its arguments' last field) of every call."""
    orc.build()
    ssm._load()
    seen, current = [], [0]

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                seen.append((current[0], name, struct.unpack(f"{len(args[-1]) // 8}q", args[-1])[-1]))
                return 0
            return entry

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before
    monkeypatch.setattr(ssm, "_lib", Library())
    monkeypatch.setattr(ssm, "_current_device", lambda: current[0])
    monkeypatch.setattr(ssm, "_one_device", False)
    monkeypatch.setattr(ssm, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


@pytest.mark.parametrize("dev", [0, 1])
def test_calls_run_on_their_tensors_device(calls, dev):
    t = lambda *s, d=torch.float32: FakeTensor(s, d, dev)  # noqa: E731
    plan = ssm.SSM(None, 8, 4, 1, 3, 1)
    X, bc, W, A = t(2, 5, 8), t(2, 5, 1, 4), t(8, 3), t(8, 4)
    orc.rnn_ssm_conv(plan, X, W, Y=X)
    orc.rnn_ssm_conv_grad(plan, X, X, W)
    orc.rnn_ssm_scan(plan, X, X, A, bc, bc, Y=X)
    orc.rnn_ssm_conv_step(plan, t(2, 8), W, None, t(2, 2, 8), t(2, 8))
    orc.rnn_ssm_scan_step(plan, t(2, 8), t(2, 8), A, t(2, 1, 4), t(2, 1, 4), t(2, 8, 4), t(2, 8))
    logits, ids = t(3, 9), t(3, d=torch.int32)
    orc.rnn_scores(logits, ids, lse=t(3))
    orc.rnn_scores_grad(logits, ids, orc.Scores(None, None, t(3), None, None), dlogits=logits)
    assert [c[1] for c in calls] == ["rnn_ssm_conv", "rnn_ssm_conv_grad", "rnn_ssm_scan", "rnn_ssm_conv_step",
                                     "rnn_ssm_scan_step", "rnn_scores", "rnn_scores_grad"]
    assert all(c[0] == dev and c[2] == 1000 + dev for c in calls)       # that device, and its current stream


def test_the_gradient_of_the_scan_too(calls):
    t = lambda *s: FakeTensor(s, torch.float32, 1)  # noqa: E731
    plan = ssm.SSM(None, 8, 4, 1, 3, 1)
    X, bc, A = t(2, 5, 8), t(2, 5, 1, 4), t(8, 4)
    plan_size = ssm.rnn_ssm_saved_size
    try:
        ssm.rnn_ssm_saved_size = lambda *a: 7
        orc.rnn_ssm_scan_grad(plan, X, t(7), X, X, A, bc, bc)
    finally:
        ssm.rnn_ssm_saved_size = plan_size
    assert calls == [(1, "rnn_ssm_scan_grad", 1001)]


def test_tensors_of_two_devices_are_refused(calls):
    plan = ssm.SSM(None, 8, 4, 1, 3, 1)
    X = FakeTensor((2, 5, 8), torch.float32, 1)
    with pytest.raises(ValueError):
        orc.rnn_ssm_conv(plan, X, FakeTensor((8, 3), torch.float32, 0), Y=X)
    assert not calls
