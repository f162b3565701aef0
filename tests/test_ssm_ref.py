"""The 64-bit references of the state space and score operators: their
gradients against torch's differentiation of the forward formulas and against
central differences, and the refusals of the entry points that need no GPU."""
import ctypes
import struct

import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref


@pytest.fixture(scope="module")
def lib():
    orc.build()
    from onnx_recurrent_gb300 import ssm
    return ssm._load()


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def _scan_case(seed, N=3, S=7, D=6, G=2, M=5):
    r = _rand(seed)
    return dict(X=r(N, S, D), dt=r(N, S, D), A=-torch.exp(r(D, M)), B=r(N, S, G, M), C=r(N, S, G, M), D=r(D),
                Z=r(N, S, D), dt_bias=r(D), h0=r(N, D, M)), r(N, S, D), r(N, D, M), torch.tensor([S, 0, S - 2])


def test_scan_gradient_is_the_forward_formulas_derivative():
    v, dY, dYh, lens = _scan_case(1)
    leaf = {k: t.clone().requires_grad_(True) for k, t in v.items()}
    Y, Yh = ref.scan(leaf["X"], leaf["dt"], leaf["A"], leaf["B"], leaf["C"], leaf["D"], leaf["Z"], leaf["dt_bias"], lens,
                     leaf["h0"])[:2]
    ((Y * dY).sum() + (Yh * dYh).sum()).backward()
    got = ref.scan_grad(dY, dYh, v["X"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["Z"], v["dt_bias"], lens, v["h0"])
    for mine, theirs in (("dX", "X"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"), ("dD", "D"), ("dZ", "Z"),
                         ("ddt_bias", "dt_bias"), ("d_initial_h", "h0")):
        assert torch.allclose(got[mine], leaf[theirs].grad, rtol=1e-10, atol=1e-12), mine


def test_conv_gradient_is_the_forward_formulas_derivative():
    r = _rand(2)
    N, S, D, K = 3, 6, 4, 4
    v = dict(X=r(N, S, D), W=r(D, K), bias=r(D), h0=r(N, K - 1, D))
    dY, dhT, lens = r(N, S, D), r(N, K - 1, D), torch.tensor([S, 0, 2])
    leaf = {k: t.clone().requires_grad_(True) for k, t in v.items()}
    Y, hT, _ = ref.conv(leaf["X"], leaf["W"], leaf["bias"], lens, leaf["h0"], True)
    ((Y * dY).sum() + (hT * dhT).sum()).backward()
    got = ref.conv_grad(dY, dhT, v["X"], v["W"], v["bias"], lens, v["h0"], True)
    for mine, theirs in (("dX", "X"), ("dW", "W"), ("dbias", "bias"), ("d_initial_state", "h0")):
        assert torch.allclose(got[mine], leaf[theirs].grad, rtol=1e-10, atol=1e-12), mine


def test_scores_gradient_matches_differences():
    r = _rand(3)
    x, ids, top = r(4, 9), torch.tensor([2, 0, -1, 8]), 3
    dl, dh, dt = r(4), r(4), r(4, top)
    f = lambda v: sum((out[k] * w).sum() for out in [ref.scores(v, ids, top)]  # noqa: E731
                      for k, w in (("logp", dl), ("entropy", dh), ("top_logp", dt)))
    g = ref.scores_grad(x, ids, ref.scores(x, ids, top), dl, dh, dt)
    eps = 1e-6
    for _ in range(5):
        d = r(4, 9)
        assert abs(float((f(x + eps * d) - f(x - eps * d)) / (2 * eps) - (g * d).sum())) < 1e-7


# ------------------------------------------------------------ refusals

@pytest.mark.parametrize("kw", [dict(channels=0), dict(channels=-4), dict(state_size=0), dict(state_size=129),
                                dict(groups=0), dict(groups=3), dict(conv_width=0), dict(conv_width=9), dict(layout=2)])
def test_create_refuses(lib, kw):
    args = dict(channels=8, state_size=16, groups=1, conv_width=4, layout=0)
    args.update(kw)
    with pytest.raises(orc.RNNError) as e:
        orc.rnn_ssm_create(**args)
    assert e.value.status == 1 and e.value.message


def test_create_refuses_activation_and_io_type(lib):
    with pytest.raises(ValueError):
        orc.rnn_ssm_create(8, activation="gelu")
    p = orc.rnn_ssm_create(8)
    with pytest.raises(orc.RNNError) as e:
        orc.rnn_ssm_set_io_type(p, 5)
    assert e.value.status == 1
    orc.rnn_ssm_destroy(p)
    orc.rnn_ssm_destroy(p)      # idempotent in the binding


def test_null_plan_and_args(lib):
    for name in ("conv", "conv_grad", "conv_step", "scan", "scan_grad", "scan_step"):
        assert getattr(lib, "rnn_ssm_" + name)(None, bytes(512)) == 1, name
        p = orc.rnn_ssm_create(8)
        assert getattr(lib, "rnn_ssm_" + name)(p.handle, None) == 1, name
        assert "args" in orc.rnn_last_error()
    assert lib.rnn_scores(None) == 1 and lib.rnn_scores_grad(None) == 1
    assert lib.rnn_ssm_saved_size(None, 4, 4) == -1


def test_runs_refuse_before_device_work(lib):
    """Arguments in the order of the header's structures; 64 stands for a pointer that must not be read."""
    p = orc.rnn_ssm_create(8, state_size=4, conv_width=3)
    conv = [5, 2, 64, 0, 0, 64, 0, 0, 0, 64, 0, 0, 0, 0]
    def run(name, fields, handle=True):  # noqa: E301
        fn = getattr(lib, name)
        raw = struct.pack(f"{len(fields)}q", *fields)
        return fn(p.handle, raw) if handle else fn(raw)
    for at, value, word in ((0, -1, "seq_length"), (1, -1, "batch_size"), (2, 0, "X"), (3, -8, "negative stride"),
                            (2, 66, "aligned"), (5, 0, "W"), (9, 0, "Y")):
        bad = list(conv)
        bad[at] = value
        assert run("rnn_ssm_conv", bad) == 1, (at, value)
        assert word in orc.rnn_last_error()
    step = [2, 0, 64, 0, 0, 64, 0, 64, 64, 64, 64, 0, 0, 0]      # slots without n_slots
    assert run("rnn_ssm_conv_step", step) == 1 and "n_slots" in orc.rnn_last_error()
    scores = [4, 10, 0, 0, 64, 0, 0, 0, 64, 64, 0, 0, 0]
    for at, value, word in ((0, -1, "rows"), (1, 0, "vocab"), (2, 5, "row_stride"), (3, 3, "io type"), (4, 0, "logits"),
                            (4, 65, "aligned"), (6, 33, "top"), (6, 11, "top"), (6, -1, "top"), (7, 64, "ids"),
                            (6, 2, "top_ids")):
        bad = list(scores)
        bad[at] = value
        assert run("rnn_scores", bad, False) == 1, (at, value)
        assert word in orc.rnn_last_error()
    assert run("rnn_scores", [0, 10] + [0] * 11, False) == 0     # no rows: nothing is read
    assert run("rnn_ssm_conv", [5, 0] + [0] * 12) == 0           # no batch: nothing is read
    assert ctypes.sizeof(ctypes.c_void_p) == 8
