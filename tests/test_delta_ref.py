"""The 64-bit references against plainer forms of themselves and against differences."""
import torch

import delta_ref64 as ref


def _case(N=2, S=5, H=4, HK=2, DK=3, DV=2):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    return (unit(r(N, S, HK, DK)), unit(r(N, S, HK, DK)), r(N, S, H, DV), -torch.rand(N, S, H, generator=g, dtype=torch.float64),
            torch.rand(N, S, H, generator=g, dtype=torch.float64)), r(N, H, DK, DV)


def test_delta_written_out_for_one_head():
    (Q, K, V, g, beta), st = _case(1, 4, 1, 1, 3, 2)
    Y, end = ref.delta(Q, K, V, g, beta, None, st, 0.5)
    S = st[0, 0]
    for t in range(4):
        k, q, a, b = K[0, t, 0], Q[0, t, 0], float(torch.exp(g[0, t, 0])), float(beta[0, t, 0])
        S = a * (torch.eye(3, dtype=torch.float64) - b * torch.outer(k, k)) @ S + b * torch.outer(k, V[0, t, 0])
        assert torch.allclose(Y[0, t, 0], 0.5 * S.T @ q, rtol=1e-13)
    assert torch.allclose(end[0, 0], S, rtol=1e-13)


def test_delta_lengths():
    (Q, K, V, g, beta), st = _case()
    lens = torch.tensor([3, 0])
    Y, end = ref.delta(Q, K, V, g, beta, lens, st, 1.0)
    short, after = ref.delta(*(t[:1, :3] for t in (Q, K, V, g, beta)), None, st[:1], 1.0)
    assert torch.equal(Y[0, :3], short[0]) and not Y[0, 3:].any() and not Y[1].any()
    assert torch.equal(end[0], after[0]) and torch.equal(end[1], st[1])


def test_delta_gradient_against_differences():
    ins, st = _case()
    lens = torch.tensor([5, 3])
    leaves = [t.clone().requires_grad_() for t in (*ins, st)]
    assert torch.autograd.gradcheck(lambda *a: ref.delta(*a[:5], lens, a[5], 0.7), leaves, atol=1e-6)


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    X, W, b = (torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_() for s in ((3, 7), (7,), (7,)))
    assert torch.autograd.gradcheck(lambda *a: ref.norm(*a, 1e-5)[0], (X, W, b))


def test_beam_by_enumeration():
    logits = torch.tensor([[[0.0, 1.0, 2.0], [2.0, 2.0, -1.0]]], dtype=torch.float64)
    scores, done = torch.tensor([[-1.0, -1.5]]), torch.tensor([[False, True]])
    parents, ids, new, fin = ref.beam(logits, scores, done, 0)
    lp = torch.log_softmax(logits[0, 0], 0)
    assert parents.tolist() == [[0, 1]] and ids.tolist() == [[2, 0]] and fin.tolist() == [[False, True]]
    assert torch.allclose(new[0], torch.tensor([float(lp[2]) - 1.0, -1.5], dtype=torch.float64))
