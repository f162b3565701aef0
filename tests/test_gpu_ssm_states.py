"""State sizes between the powers of two that have a test of their own, runs
split over their steps with more than 16 states, and errors as norms, which
a bound for every step's worst rounding would let pass."""
import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref
from test_gpu_ssm import DT, _check_scan, _d, _scan_case, _scan_run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


STATES = [  # N, S, D, M, G, io, layout, lens, carried, gate, skip, soft
    (2, 20, 37, 17, 1, "f32", 1, True, True, True, True, True),
    (3, 33, 66, 20, 3, "bf16", 0, True, True, True, True, True),
    (2, 18, 70, 24, 1, "f16", 1, None, False, True, False, True),
    (8, 35, 64, 32, 2, "f32", 0, True, True, True, True, True),
    (2, 31, 24, 31, 1, "f32", 1, True, True, False, True, False),
    (1, 160, 136, 32, 1, "f32", 1, None, True, True, True, True),      # split
    (2, 500, 40, 24, 2, "bf16", 0, True, True, True, True, True),
    (2, 400, 24, 64, 1, "f32", 1, True, True, True, True, True),
    (1, 300, 20, 128, 1, "f16", 1, None, True, True, True, True),
    (2, 260, 30, 33, 1, "f32", 0, True, False, True, True, True),
]


@pytest.mark.parametrize("c", STATES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("views", [False, True])
def test_scan_and_gradient(c, views):
    v, dY, dYh, ln = _scan_case(c)
    _check_scan(c, v, dY, dYh, ln, _scan_run(c, v, dY, dYh, ln, views))


@pytest.mark.parametrize("N,D,M,G,io", [(2, 37, 17, 1, "f32"), (5, 66, 20, 3, "f16"), (70, 40, 32, 2, "bf16"), (3, 24, 24, 1, "f32"),
                                        (40, 1024, 32, 1, "bf16")])
def test_scan_step(N, D, M, G, io):
    c = (N, 1, D, M, G, io, 1, None, True, True, True, True)
    v, _, _, _ = _scan_case(c, seed=2)
    cu = {k: t.cuda() for k, t in v.items()}
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G)
    orc.rnn_ssm_set_io_type(plan, io)
    Y, out = torch.empty(N, D, dtype=DT[io], device="cuda"), torch.empty(N, D, M, device="cuda")
    orc.rnn_ssm_scan_step(plan, cu["X"][:, 0], cu["dt"][:, 0], cu["A"], cu["B"][:, 0], cu["C"][:, 0], cu["h0"], Y, cu["D"],
                          cu["Z"][:, 0], cu["dt_bias"], H_out=out)
    d = {k: _d(t) for k, t in v.items()}
    a = (d["X"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["Z"], d["dt_bias"], None, d["h0"])
    rY, rH, _, _, delta, _ = ref.scan(*a)
    mY, mH = ref.scan(*a, magnitude=True)[:2]
    u = ref.steps_bound(1, M, float((delta[..., None] * d["A"].abs()).max()))
    ref.close(Y, rY[:, 0], u * mY[:, 0], io, "Y")
    ref.close(out, rH, u * mH, "f32", "H")


NORMS = [(1, 1100, 32, 16, 1), (3, 300, 64, 16, 2), (2, 400, 40, 24, 1), (1, 300, 136, 64, 1), (64, 260, 512, 16, 1)]


@pytest.mark.parametrize("size", NORMS, ids=lambda c: "-".join(map(str, c)))
def test_errors_as_norms(size):
    """fp32 throughout.  Here delta |A| is above 0.02 for all but a few channels and states, so a state remembers at most 50 steps: a
    decay off by up to 0.5 u to one side leaves it 25 u off; roundings of random sign (a state's over its memory, sums over up to 64
    states, the gate) add less than 16 u.  A gradient passes the states' memory and its own and one
    sum more: 128 u."""
    N, S, D, M, G = size
    c = (N, S, D, M, G, "f32", 1, None, True, True, True, True)
    v, dY, dYh, _ = _scan_case(c, seed=11)
    got = _scan_run(c, v, dY, dYh, None)
    cu = {k: _d(t) for k, t in v.items()}
    a = (cu["X"], cu["dt"], cu["A"], cu["B"], cu["C"], cu["D"], cu["Z"], cu["dt_bias"])
    if N > 4:                                 # the last row stands for all, but for sums over the rows
        a = tuple(t[-1:] if t.dim() > 2 else t for t in a)
    h0 = cu["h0"][-1:] if N > 4 else cu["h0"]
    n = slice(-1, None) if N > 4 else slice(None)
    Y, Yh = ref.scan(*a, None, h0)[:2]
    off = lambda g, w: float((g.double().cpu() - w).norm() / w.norm()) / ref.U  # noqa: E731
    assert off(got["Y"][n], Y) <= 64 and off(got["Y_h"][n], Yh) <= 64
    want = ref.scan_grad(_d(dY)[n], _d(dYh)[n], *a, None, h0)
    for k, w in want.items():
        if N > 4 and k in ("dA", "dD", "ddt_bias"):
            continue
        assert off(got[k][n] if w.dim() > 2 else got[k], w) <= 128, k
