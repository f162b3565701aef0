"""What the differentiable functions do besides a first gradient: second
derivatives, outputs that a loss leaves out, inputs that need no gradient."""
import pytest
import torch

import onnx_recurrent_gb300 as orc
from onnx_recurrent_gb300 import autograd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).cuda()


def _layer(seed=0, N=2, S=9, D=8, M=4):
    r = _rand(seed)
    plan = orc.rnn_ssm_create(D, state_size=M, layout=1)
    v = dict(X=r(N, S, D), dt=r(N, S, D, scale=0.5), A=-torch.exp(r(D, M)), B=r(N, S, 1, M), C=r(N, S, 1, M), D=r(D),
             Z=r(N, S, D), dt_bias=r(D) - 2, initial_h=r(N, D, M))
    return plan, v, dict(W=r(D, 4), bias=r(D), initial_state=r(N, 3, D))


def _leaves(v):
    return {k: t.clone().requires_grad_(True) for k, t in v.items()}


@pytest.mark.parametrize("which", ["conv", "scan", "scores"])
def test_second_derivatives_are_refused(which):
    plan, v, c = _layer()
    x = v["X"].clone().requires_grad_(True)
    if which == "conv":
        out = autograd.conv(plan, x ** 3, **c)[0]
    elif which == "scan":
        out = autograd.scan(plan, x ** 3, **{k: t for k, t in v.items() if k != "X"})[0]
    else:
        ids = torch.zeros(18, dtype=torch.int32, device="cuda")
        out = autograd.scores((x ** 3).reshape(18, 8), ids)[0]
    g, = torch.autograd.grad(out.square().sum(), x, create_graph=True)      # a gradient penalty's first half
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


@pytest.mark.parametrize("top", [0, 3])
def test_scores_without_tokens(top):
    """A loss of the entropy and the alternatives alone."""
    r = _rand(1)
    x = r(7, 50).requires_grad_(True)
    out = autograd.scores(x, top=top)
    assert out[0] is None and len(out) == (4 if top else 2)
    w = r(7), r(7, 3)
    loss = (out[1] * w[0]).sum() + ((out[3] * w[1]).sum() if top else 0)
    loss.backward()
    y = x.detach().double().requires_grad_(True)
    logp = torch.log_softmax(y, 1)
    want = (-(logp.exp() * logp).sum(1) * w[0]).sum()
    if top:
        want = want + (logp.topk(3).values * w[1]).sum()
    want.backward()
    # products of a few roundings each, of terms below 4 in all: as a norm
    assert float((x.grad - y.grad).norm() / y.grad.norm()) <= 1e-6


def _grads(fn, plan, v, use):
    leaf = _leaves(v)
    outs = fn(plan, **leaf)
    r = _rand(3)
    sum((o * r(*o.shape)).sum() * u for o, u in zip(outs, use)).backward()
    return {k: t.grad for k, t in leaf.items()}


@pytest.mark.parametrize("used", [0, 1])
def test_a_loss_of_one_output(used):
    """The other's slopes are zeros, whether a tensor holds them or none does."""
    plan, v, c = _layer(4)
    c["X"] = v["X"]
    for fn, inputs in ((autograd.scan, v), (autograd.conv, c)):
        leaf = _leaves(inputs)
        outs = fn(plan, **leaf)
        w = _rand(5)(*outs[used].shape)
        (outs[used] * w).sum().backward()
        full = _leaves(inputs)
        outs = fn(plan, **full)
        ((outs[used] * w).sum() + (outs[1 - used] * 0).sum()).backward()
        for k in inputs:
            assert torch.equal(leaf[k].grad, full[k].grad), k


@pytest.mark.parametrize("which", ["scan", "conv"])
def test_only_the_gradients_asked_for(which):
    plan, v, c = _layer(6)
    c["X"] = v["X"]
    fn, inputs = (autograd.scan, v) if which == "scan" else (autograd.conv, c)
    want = _grads(fn, plan, inputs, (1, 1))
    for name in inputs:
        one = {k: t.clone().requires_grad_(k == name) for k, t in inputs.items()}
        outs = fn(plan, **one)
        r = _rand(3)
        sum((o * r(*o.shape)).sum() for o in outs).backward()
        assert torch.equal(one[name].grad, want[name]), name
        assert all(t.grad is None for k, t in one.items() if k != name)


@pytest.mark.parametrize("off", ["no_grad", "inference_mode", "no leaf"])
def test_a_scan_without_gradients_saves_nothing(off):
    """What the states and y would take on top of the outputs is not allocated."""
    N, S, D, M = 2, 512, 256, 16
    plan, v, _ = _layer(7, N, S, D, M)
    if off != "no leaf":
        v = _leaves(v)
    saved = orc.rnn_ssm_saved_size(plan, S, N) * 4
    outputs = 4 * (N * S * D + N * D * M)

    def peak():
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        with torch.no_grad() if off == "no_grad" else torch.inference_mode(off == "inference_mode"):
            Y, Y_h = autograd.scan(plan, **v)
        assert not Y.requires_grad
        return torch.cuda.max_memory_allocated() - before, Y, Y_h
    taken, Y, Y_h = peak()
    assert saved > outputs and taken < outputs + saved // 2
    want = orc.ssm_scan(plan, **{k: t.detach() for k, t in v.items()})
    assert torch.equal(Y, want[0]) and torch.equal(Y_h, want[1])
