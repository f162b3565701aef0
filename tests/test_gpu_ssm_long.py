"""Long memories: a state that remembers thousands of steps adds up what every
decay is off by, if that is always to the same side.

Bounds.  u = 2^-24.  A state of decay exp(-r) remembers 1 / r steps.  An error of
b u in each decay, always to one side, leaves the state b u / r off; errors of
random sign, of a root mean square of e u a step, e u / sqrt(2 r).  b <= 0.04 is what the
correction of the hardware's 2^x leaves for r below 0.002; e < 1.1 (2^x's own 0.5 u, half
a unit in the last place each for its argument and the update).  The steps differ from token to
token, as a model's do: the same step each time would round the same way each time.
The norm of the difference over the norm of the states is then below
(0.04 / r + 1.1 / sqrt(2 r)) u with r the smallest of all rates."""
import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


def _case(M, rate, S, D, seed):
    """One row: rates of 0.75 to 1.25 times `rate`, steps of half to one and a half times that."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    delta = (rate * (0.5 + torch.rand(1, S, D, generator=g))).cuda()
    A = -(0.75 + 0.5 * torch.rand(D, M, generator=g)).cuda()
    return dict(X=1 + r(1, S, D), dt=delta, A=A, B=1 + 0.5 * r(1, S, 1, M), C=r(1, S, 1, M)), r(1, D, M).abs() + 0.5


def _states(v, h):
    h = h.double()
    for t in range(v["X"].shape[1]):
        d = v["dt"][:, t].double()
        h = torch.exp(d[..., None] * v["A"].double()) * h + (d * v["X"][:, t].double())[..., None] * v["B"][:, t].double()
    return h


def _bound(rate):
    r = 0.75 * rate
    return (0.04 / r + 1.1 / (2 * r) ** 0.5) * ref.U


# states that a vector access takes and states that it does not, more than 16 of them
@pytest.mark.parametrize("M,rate,S", [(16, 1e-3, 4000), (16, 3e-4, 12000), (6, 1e-3, 4000), (20, 5e-4, 6000), (32, 1e-3, 4000)])
def test_a_state_taken_token_by_token(M, rate, S):
    v, h0 = _case(M, rate, S, 64, seed=M)
    plan = orc.rnn_ssm_create(64, state_size=M, softplus=False)
    h, y = h0.clone(), torch.empty_like(v["X"][:, 0])
    for t in range(S):
        orc.rnn_ssm_scan_step(plan, v["X"][:, t], v["dt"][:, t], v["A"], v["B"][:, t], v["C"][:, t], h, y)
    want = _states(v, h0)
    assert float((h - want).norm() / want.norm()) <= _bound(rate)


@pytest.mark.parametrize("M,rate,S", [(16, 1e-3, 3000), (20, 1e-3, 3000), (16, 5e-4, 3000)])
def test_a_state_taken_by_the_scan_unsplit(M, rate, S):
    """Rows enough to fill the SMs (all of them the same): every state passes all steps in one block."""
    N, D = 152, 512
    v, h0 = _case(M, rate, S, D, seed=M + 1)
    plan = orc.rnn_ssm_create(D, state_size=M, softplus=False, layout=1)
    rows = {k: t if k == "A" else t.expand(N, *t.shape[1:]) for k, t in v.items()}
    _, h, _ = orc.ssm_scan(plan, **rows, initial_h=h0.repeat(N, 1, 1))
    assert orc.rnn_ssm_last_launch_count(plan) == 1
    want = _states(v, h0)
    assert torch.equal(h[:1], h[-1:])
    assert float((h[:1] - want).norm() / want.norm()) <= _bound(rate)


@pytest.mark.parametrize("M,rate,S", [(16, 1e-3, 4000), (20, 5e-4, 6000), (32, 1e-3, 4000)])
def test_a_state_taken_by_the_scan_split(M, rate, S):
    v, h0 = _case(M, rate, S, 64, seed=M + 2)
    plan = orc.rnn_ssm_create(64, state_size=M, softplus=False, layout=1)
    _, h, _ = orc.ssm_scan(plan, **v, initial_h=h0)
    assert orc.rnn_ssm_last_launch_count(plan) > 1
    want = _states(v, h0)
    assert float((h - want).norm() / want.norm()) <= _bound(rate)
