"""The operators together: the differentiable functions against the references,
and the example's model trained a little and continued token by token."""
import os
import sys

import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref
from onnx_recurrent_gb300 import autograd

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import ssm_language_model
    return ssm_language_model


def test_functions_chain_like_the_references():
    """scores(conv -> scan -> product) in fp32: every leaf's gradient against 64-bit differentiation."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).double()  # noqa: E731
    N, S, D, M, V = 2, 19, 12, 16, 33
    leaf = dict(x=r(N, S, D), W=r(D, 4, scale=0.5), b=r(D), dt=r(N, S, D, scale=0.5), A=-torch.exp(r(D, M, scale=0.5)),
                B=r(N, S, 1, M), C=r(N, S, 1, M), skip=r(D), z=r(N, S, D), bias=r(D, scale=0.5) - 2, head=r(D, V, scale=0.3),
                h0=r(N, D, M), c0=r(N, 3, D))
    ids = torch.randint(0, V, (N * S,), generator=g, dtype=torch.int32)

    def reference(v):
        u = ref.conv(v["x"], v["W"], v["b"], None, v["c0"], True)[0]
        y = ref.scan(u, v["dt"], v["A"], v["B"], v["C"], v["skip"], v["z"], v["bias"], None, v["h0"])[0]
        lp = torch.log_softmax((y.reshape(-1, D) @ v["head"]), -1)
        return -(lp.gather(1, ids.long()[:, None]).mean()) + 0.1 * (lp.exp() * lp).sum(-1).mean()
    a = {k: t.clone().requires_grad_(True) for k, t in leaf.items()}
    want = reference(a)
    want.backward()
    plan = orc.rnn_ssm_create(D, state_size=M, layout=1)
    b = {k: t.float().cuda().requires_grad_(True) for k, t in leaf.items()}
    u, _ = autograd.conv(plan, b["x"], b["W"], b["b"], None, b["c0"])
    y, _ = autograd.scan(plan, u, b["dt"], b["A"], b["B"], b["C"], b["skip"], b["z"], b["bias"], None, b["h0"])
    logp, entropy = autograd.scores(y.reshape(-1, D) @ b["head"], ids.cuda())
    got = -logp.mean() - 0.1 * entropy.mean()
    got.backward()
    assert abs(float(got) - float(want)) < 1e-5 * abs(float(want))
    for k in leaf:
        scale = a[k].grad.abs().max()
        assert float((b[k].grad.cpu().double() - a[k].grad).abs().max()) <= 2e-5 * float(scale), k


def test_example_learns_and_continues(example):
    torch.manual_seed(0)
    model = example.Model(width=32, inner=64, layers=2, io="bf16").cuda()
    losses = example.train(model, 25, batch=16, length=32)
    assert losses[-1] < 0.8 * losses[0]
    prompt = [0, 1, 5, 2]
    ids, logps, others = example.generate(model, prompt, 10)
    assert len(ids) == 14 and all(lp <= 0 for lp in logps) and all(len(o) == 2 for o in others)
    for layer in model.layers:
        orc.rnn_ssm_sync(layer.plan)


def test_example_tokens_match_the_whole_sequence(example):
    """A prompt's logits by the whole-sequence operators and token by token (fp32)."""
    torch.manual_seed(1)
    model = example.Model(width=32, inner=64, layers=2, io="f32").cuda()
    ids = torch.randint(0, 9, (2, 14), device="cuda")
    with torch.no_grad():
        whole, _ = model(ids)
        logits, states = model(ids[:, :6])
        parts = [logits[:, -1]]
        for t in range(6, 14):
            parts.append(model.step(ids[:, t], states))
    got = torch.stack(parts, 1)
    assert torch.allclose(got, whole[:, 5:], rtol=1e-4, atol=1e-4)
