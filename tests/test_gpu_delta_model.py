"""The gated delta rule, layer normalisation, scores and beam search together, as a model uses them: the
differentiable functions against 64-bit differentiation and differences, the example's model, and a captured token.

Bounds: the delta rule's outputs and gradients err by 4 sqrt(S (DK + 128)) u of their norm (see delta_ref64), a
normalisation's or the scores' by a few u; each operator passes the errors of the one before it on with a factor near 1
(rows of unit variance, keys of length 1), two to each side of the differentiation: in all 4 times the first."""
import itertools
import os
import sys

import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc
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


def _inputs(seed=0, N=2, S=70, H=4, HK=2, DK=16, DV=24):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    v = dict(Q=0.99 * unit(r(N, S, HK, DK)), K=0.99 * unit(r(N, S, HK, DK)), V=r(N, S, H, DV), g=-r(N, S, H).abs() * 0.3,
             beta=torch.sigmoid(r(N, S, H)), initial_state=r(N, H, DK, DV))
    return g, {k: t.float().double() for k, t in v.items()}


def _plan(v, layout=1):
    return orc.rnn_delta_create(v["V"].shape[2], v["Q"].shape[3], v["V"].shape[3], v["Q"].shape[2], layout=layout)


def _leaves(v, **only):
    return {k: t.float().cuda().requires_grad_(only.get(k, not only)) for k, t in v.items()}


def test_functions_chain_like_the_references():
    """scores(norm(delta(norm(x))) @ head): every leaf's gradient against 64-bit differentiation."""
    gen, v = _inputs()
    N, S, H, DV = v["V"].shape
    D, vocab = H * DV, 33
    r = lambda *s: torch.randn(*s, generator=gen).double()  # noqa: E731
    v.update(w1=1 + 0.1 * r(DV), w2=1 + 0.1 * r(D), b2=0.1 * r(D), head=r(D, vocab) * 0.2)
    ids = torch.randint(0, vocab, (N * S,), generator=gen, dtype=torch.int32)
    plan = _plan(v)
    first, second = orc.rnn_norm_create(DV), orc.rnn_norm_create(D)

    def reference(a):
        x = torch.nn.functional.layer_norm(a["V"], (DV,), a["w1"])
        y, state = ref.delta(a["Q"], a["K"], x, a["g"], a["beta"], None, a["initial_state"], plan.scale)
        h = torch.nn.functional.layer_norm(y.reshape(-1, D), (D,), a["w2"], a["b2"])
        lp = torch.log_softmax(h @ a["head"], -1)
        return -lp.gather(1, ids.long()[:, None]).mean() + 0.1 * (lp.exp() * lp).sum(-1).mean() + 0.01 * (state * state).mean()
    a = {k: t.clone().requires_grad_(True) for k, t in v.items()}
    want = reference(a)
    want.backward()
    b = _leaves(v)
    x = autograd.layer_norm(first, b["V"], b["w1"])
    y, state = autograd.delta_rule(plan, b["Q"], b["K"], x, b["g"], b["beta"], None, b["initial_state"])
    h = autograd.layer_norm(second, y.flatten(0, 1).flatten(1), b["w2"], b["b2"])
    logp, entropy = autograd.scores(h @ b["head"], ids.cuda())
    got = -logp.mean() - 0.1 * entropy.mean() + 0.01 * (state * state).mean()
    got.backward()
    bound = 4 * 4 * (S * (v["Q"].shape[3] + 128)) ** 0.5 * ref.U
    assert abs(float(got.detach()) - float(want.detach())) <= bound * abs(float(want.detach()))
    for k in v:
        err = (b[k].grad.cpu().double() - a[k].grad).norm() / a[k].grad.norm()
        assert float(err) <= bound, (k, float(err))


@pytest.mark.parametrize("name", ["Q", "K", "V", "g", "beta", "initial_state"])
def test_delta_gradients_against_differences(name):
    """The slope along the gradient's own direction d (of length 1), which is its length, from f = sum w Y + sum w' state at four
    points: (8 (f1 - f-1) - (f2 - f-2)) / 12 h, here with h = 0.02.  That errs by h^4 f5 / 30, below 1e-6 ||w|| ||Y|| for
    changes of unit length; by 18 E / 12 h = 75 E, E the error of f: the weights are drawn independently of the outputs'
    errors e, so sum w e is below 5 ||e|| (five deviations), ||e|| <= 4 sqrt(S (DK + 128)) u ||Y||; and by 75 |slope| u ||input|| for
    the rounding of the moved inputs."""
    gen, v = _inputs(3)
    S = v["V"].shape[1]
    plan, order = _plan(v), ("Q", "K", "V", "g", "beta")
    w = [torch.randn(*s, generator=gen).double() for s in (v["V"].shape, v["initial_state"].shape)]
    b = _leaves(v, **{name: True})
    outs = autograd.delta_rule(plan, *(b[k] for k in order), None, b["initial_state"])
    sum((o * x.float().cuda()).sum() for o, x in zip(outs, w)).backward()
    grad = b[name].grad.cpu().double()
    got = float(grad.norm())

    def f(h):
        a = {k: t.float().cuda() for k, t in v.items()}
        a[name] = (v[name] + h * grad / got).float().cuda()
        moved = autograd.delta_rule(plan, *(a[k] for k in order), None, a["initial_state"])
        return sum(float((o.cpu().double() * x).sum()) for o, x in zip(moved, w))
    h = 0.02
    want = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    Y = sum(float(o.detach().norm()) for o in outs)
    E = 5 * 4 * (S * (v["Q"].shape[3] + 128)) ** 0.5 * ref.U * Y
    bound = 75 * E + 1e-6 * Y * sum(float(x.norm()) for x in w) + 75 * got * ref.U * float(v[name].norm())
    assert abs(got - want) <= bound and bound < 0.05 * got


@pytest.mark.parametrize("which", ["delta", "norm"])
def test_second_derivatives_are_refused(which):
    _, v = _inputs(1, S=9)
    x = v["V"].float().cuda().requires_grad_(True)
    if which == "delta":
        a = {k: t.float().cuda() for k, t in v.items()}
        out = autograd.delta_rule(_plan(v), a["Q"], a["K"], x ** 3, a["g"], a["beta"])[0]
    else:
        out = autograd.layer_norm(orc.rnn_norm_create(x.shape[-1]), x ** 3)
    g, = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()


@pytest.mark.parametrize("used", [0, 1])
@pytest.mark.parametrize("layout", [0, 1])
def test_a_loss_of_one_output(used, layout):
    _, v = _inputs(4)
    if layout == 0:
        v = {k: t if k == "initial_state" else t.transpose(0, 1).contiguous() for k, t in v.items()}
    plan, order = _plan(v, layout), ("Q", "K", "V", "g", "beta")
    grads = []
    for also in (False, True):
        b = _leaves(v)
        outs = autograd.delta_rule(plan, *(b[k] for k in order), None, b["initial_state"])
        loss = outs[used].square().sum()
        (loss + (outs[1 - used] * 0).sum() if also else loss).backward()
        grads.append({k: t.grad for k, t in b.items()})
    for k in v:
        assert torch.equal(grads[0][k], grads[1][k]), k


@pytest.mark.parametrize("name", ["Q", "K", "V", "g", "beta", "initial_state"])
def test_only_the_gradients_asked_for(name):
    _, v = _inputs(6)
    plan, order = _plan(v), ("Q", "K", "V", "g", "beta")
    b, one = _leaves(v), _leaves(v, **{name: True})
    for leaf in (b, one):
        outs = autograd.delta_rule(plan, *(leaf[k] for k in order), None, leaf["initial_state"])
        sum(o.square().sum() for o in outs).backward()
    assert torch.equal(one[name].grad, b[name].grad)
    assert all(t.grad is None for k, t in one.items() if k != name)


@pytest.mark.parametrize("name", ["X", "W", "bias"])
def test_only_the_norm_gradients_asked_for(name):
    g = torch.Generator().manual_seed(0)
    v = {k: torch.randn(*s, generator=g) for k, s in (("X", (3, 5, 40)), ("W", (40,)), ("bias", (40,)))}
    plan = orc.rnn_norm_create(40)
    b = {k: t.cuda().requires_grad_() for k, t in v.items()}
    one = {k: t.cuda().requires_grad_(k == name) for k, t in v.items()}
    for leaf in (b, one):
        # a slope that is a view of another order
        autograd.layer_norm(plan, **leaf).transpose(0, 1).square().sum().backward()
    assert torch.equal(one[name].grad, b[name].grad)
    assert all(t.grad is None for k, t in one.items() if k != name)


def test_a_delta_rule_without_gradients_saves_nothing():
    _, v = _inputs(7, S=512)
    plan = _plan(v)
    b = _leaves(v)
    order = ("Q", "K", "V", "g", "beta")
    need = orc.rnn_delta_saved_size(plan, 512, 2) * 4
    autograd.delta_rule(plan, *(b[k].detach() for k in order))      # (scratch is the library's own)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with torch.no_grad():
        Y, state = autograd.delta_rule(plan, *(b[k] for k in order), None, b["initial_state"])
    taken = torch.cuda.max_memory_allocated() - before
    outputs = 4 * (Y.numel() + state.numel())
    assert not Y.requires_grad and taken < outputs + need // 2


@pytest.mark.parametrize("kinds", [["delta"], ["scan", "delta"]])
def test_example_trains_and_continues(example, kinds):
    torch.manual_seed(0)
    model = example.Model(width=32, inner=64, layers=kinds, io="bf16").cuda()
    losses = example.train(model, 5, batch=8, length=80)
    assert all(l == l for l in losses) and all(p.grad is not None and bool(p.grad.isfinite().all()) for p in model.parameters())
    ids, logps, others = example.generate(model, [0, 1, 5, 2], 6)
    assert len(ids) == 10 and all(lp <= 0 for lp in logps)


def test_example_tokens_match_the_whole_sequence(example):
    """A prompt's logits by the whole-sequence operators and token by token (fp32): both sides within the
    operators' bounds, through two layers whose inputs are normalised: 1e-4 as for the scan's layers."""
    torch.manual_seed(1)
    model = example.Model(width=32, inner=64, layers=["delta", "scan", "delta"], io="f32").cuda()
    ids = torch.randint(0, 9, (2, 80), device="cuda")
    with torch.no_grad():
        whole, _ = model(ids)
        logits, states = model(ids[:, :66])
        parts = [logits[:, -1]]
        for t in range(66, 80):
            parts.append(model.step(ids[:, t], states))
    got = torch.stack(parts, 1)
    assert torch.allclose(got, whole[:, 65:], rtol=1e-4, atol=1e-4)


def test_beams_carry_their_states(example):
    """Every beam's score is that of its tokens in the whole-sequence model, and of two tokens the best are found
    (9 beams hold every first token)."""
    torch.manual_seed(2)
    model = example.Model(width=32, inner=64, layers=["delta", "scan"], io="f32").cuda()
    prompt, words = [0, 1, 5], len(example.WORDS)

    def score(ids):
        """Of one continuation, until its full stop."""
        with torch.no_grad():
            lp = torch.log_softmax(model(torch.tensor([prompt + ids], device="cuda"))[0][0].double(), -1)
        total = 0.0
        for t, i in enumerate(ids):
            total += float(lp[len(prompt) + t - 1, i])
            if i == 8:
                break
        return total
    got, scores = example.search(model, prompt, 7, 9)
    for ids, s in zip(got.tolist(), scores.tolist()):
        stop = ids.index(8) if 8 in ids else len(ids)
        assert all(i == 8 for i in ids[stop:])
        assert abs(s - score(ids)) <= 1e-4 * 7
    assert sorted(scores.tolist(), reverse=True) == scores.tolist() and len({tuple(i) for i in got.tolist()}) == 9
    got, scores = example.search(model, prompt, 2, 9)
    every = sorted((score(list(p)) for p in itertools.product(range(words), repeat=2) if p[0] != 8 or p[1] == 8), reverse=True)
    assert torch.allclose(scores.cpu().double(), torch.tensor(every[:9], dtype=torch.float64), atol=2e-4)


def test_a_captured_token_of_a_search():
    """Normalisation, delta step, product, selection and reordering of states in one graph, replayed."""
    g = torch.Generator().manual_seed(5)
    N, B, H, DK, DV, vocab = 3, 4, 2, 16, 24, 50
    rows, D = N * B, 2 * 24
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    norm, plan, beams = orc.rnn_norm_create(D), orc.rnn_delta_create(H, DK, DV, 1, layout=1), orc.rnn_beam_create(B, end_id=3)
    table, head, w, b = r(vocab, D), r(D, vocab) * 0.3, r(D), r(D)
    q, k = (torch.nn.functional.normalize(r(rows, 1, DK), dim=-1) for _ in range(2))
    decay, beta = -r(rows, H).abs(), torch.sigmoid(r(rows, H))
    start = r(rows, H, DK, DV)

    class Run:
        def __init__(self):
            self.state, self.ids = start.clone(), torch.zeros(N, B, dtype=torch.int32, device="cuda")
            self.parents = torch.zeros_like(self.ids)
            self.scores, self.done = torch.zeros(N, B, device="cuda"), torch.zeros(N, B, dtype=torch.bool, device="cuda")
            self.x, self.y = torch.empty(rows, D, device="cuda"), torch.empty(rows, H, DV, device="cuda")

        def token(self):
            orc.rnn_layer_norm(norm, table[self.ids.flatten().long()], w, b, self.x)
            orc.rnn_delta_step(plan, q, k, self.x.unflatten(-1, (H, DV)), decay, beta, self.state, self.y)
            orc.rnn_beam_select(beams, self.y.flatten(1) @ head, self.scores, self.done, self.parents, self.ids, self.scores, self.done)
            orc.rnn_beam_reorder(beams, self.parents, [self.state])
    eager, replayed = Run(), Run()
    steps = 6
    out = []
    for _ in range(steps):
        eager.token()
        out.append((eager.ids.clone(), eager.parents.clone(), eager.scores.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.token()                    # (what the product needs on its first use)
    torch.cuda.synchronize()
    replayed.__init__()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.token()
    for ids, parents, scores in out:
        graph.replay()
        assert torch.equal(replayed.ids, ids) and torch.equal(replayed.parents, parents) and torch.equal(replayed.scores, scores)
    assert torch.equal(replayed.state, eager.state)
    orc.rnn_delta_sync(plan)
    orc.rnn_beam_sync(beams)
