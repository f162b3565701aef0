"""Token scores of rows far from zero, and of rows masked by a type's lowest
value, against 64 bits: neither a log probability nor an entropy depends on
what is added to all of a row's logits.

Bounds.  u = 2^-24.  A log probability is d log 2 - log s with |d log 2| and
log s of the order of 8 for the rows below: d's one rounding, that of log s and
that of the result are at most half a unit in the last place of a number up to 16 or
8, each evenly spread, so their root mean square is at most 16 u / sqrt(3) * (log 2 + 1/2 + 1/2)
/ 2 < 8 u together; the relative errors of s (2^x within 2 units in its last place, the
sums' roundings) add less than 4 u.  12 u bounds the root mean square over rows.  An entropy
is the difference of two such quotients and sums: 20 u."""
import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


def _exact(x, ids):
    logp = torch.log_softmax(x.double(), 1)
    return logp.gather(1, ids.long()[:, None])[:, 0], -(logp.exp() * logp).nan_to_num(0.0).sum(1), x.double().logsumexp(1)


def _rms(v):
    return float(v.double().pow(2).mean().sqrt())


@pytest.mark.parametrize("V", [40, 700, 5000, 20000])
@pytest.mark.parametrize("offset", [0.0, 30.0, -100.0, 1e3, 1e5, -1e7, 4194300.0, -1497613952.0, 2.0e9])
def test_offset_rows(V, offset):
    g = torch.Generator().manual_seed(int(abs(offset)) % 1000 + V)
    rows = 256
    # a spread of 2 around the offset, or of a few units in the offset's last place
    x = (torch.randn(rows, V, generator=g) * max(2.0, 2e-7 * abs(offset))).double().add(offset).float().cuda()
    x = x + (x == 0) * 0.5
    ids = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()
    keep = torch.log_softmax(x.double(), 1).gather(1, ids.long()[:, None])[:, 0] > -16
    ids = torch.where(keep, ids, x.argmax(1).int())
    got = orc.scores(x, ids, top=1)
    logp, entropy, lse = _exact(x, ids)
    assert _rms(got.logp - logp) <= 12 * ref.U
    assert _rms(got.entropy - entropy) <= 20 * ref.U
    assert _rms(got.top_logp[:, 0] - torch.log_softmax(x.double(), 1).max(1).values) <= 12 * ref.U
    # lse: a rounding at its own size besides
    assert float((got.lse.double() - lse).abs().max()) <= (64 + 2 * float(lse.abs().max())) * ref.U
    assert torch.equal(orc.scores(x, ids).logp, got.logp)


@pytest.mark.parametrize("low", [-1497613952.0, -2.0e9, -3.4e38, -1e6, -5e4])
@pytest.mark.parametrize("V", [1024, 20480])
def test_pieces_far_below_the_others(low, V):
    """Threads that meet far lower logits first, in the same and in other pieces: those add nothing."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(8, V, generator=g) * 2
    x[:4, :V // 2] = (low + (torch.arange(V // 2) % 3).double() * 1e-7 * abs(low)).float()
    x[4:, ::3] = low
    ids = torch.tensor([V - 1, V // 2, V - 5, V - 9, 1, 2, 4, 5], dtype=torch.int32)
    got = orc.scores(x.cuda(), ids.cuda(), top=3)
    logp, entropy, lse = _exact(x, ids)
    assert float((got.logp.cpu() - logp).abs().max()) <= 48 * ref.U
    assert float((got.entropy.cpu() - entropy).abs().max()) <= 80 * ref.U
    assert float((got.lse.cpu() - lse).abs().max()) <= 48 * ref.U
    # the log probability of a masked token
    low_ids = torch.zeros(8, dtype=torch.int32)
    logp = _exact(x, low_ids)[0]
    assert float(((orc.scores(x.cuda(), low_ids.cuda()).logp.cpu() - logp) / logp).abs().max()) <= 8 * ref.U


@pytest.mark.parametrize("io", list(DT))
@pytest.mark.parametrize("V", [1, 7, 300, 9000, 40000])
def test_rows_masked_by_the_lowest_value(io, V):
    """A row of nothing but the type's lowest value: an even row."""
    x = torch.full((3, V), torch.finfo(DT[io]).min, dtype=DT[io], device="cuda")
    ids = torch.tensor([0, V // 2, V - 1], dtype=torch.int32, device="cuda")
    got = orc.scores(x, ids, top=min(V, 4))
    want = -torch.log(torch.tensor(float(V), dtype=torch.float64))
    for v in (got.logp, got.top_logp, -got.entropy):
        assert float((v.double().cpu() - want).abs().max()) <= 48 * ref.U
    assert float(((got.lse.double().cpu() - (x.double().cpu()[0, 0] - want)) / got.lse.double().cpu()).abs().max()) <= 2 * ref.U


@pytest.mark.parametrize("io", list(DT))
@pytest.mark.parametrize("V", [5, 640, 30000])
def test_certain_tokens(io, V):
    """A log probability is never positive, and near zero as exact as fp32 sums allow."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(300, V, generator=g) * 2
    ids = torch.randint(0, V, (300,), generator=g, dtype=torch.int32)
    x[torch.arange(300), ids.long()] = torch.linspace(5, 60, 300)
    x = x.to(DT[io])
    got = orc.scores(x.cuda(), ids.cuda(), top=1)
    logp, entropy, _ = _exact(x, ids)
    assert float(got.logp.max()) <= 0 and float(got.top_logp.max()) <= 0
    sure = logp > -0.5
    assert sure.any() and float((got.logp.cpu() - logp).abs()[sure].max()) <= 16 * ref.U
    assert float((got.entropy.cpu() - entropy).abs()[sure].max()) <= 48 * ref.U


def _exact_grad(x, ids, dl, dh):
    x = x.double().requires_grad_(True)
    logp = torch.log_softmax(x, 1)
    entropy = -(logp.exp() * logp).nan_to_num(0.0).sum(1)
    loss = (logp.gather(1, ids.long()[:, None])[:, 0] * dl.double()).sum() + (entropy * dh.double()).sum()
    return torch.autograd.grad(loss, x)[0]


@pytest.mark.parametrize("V", [40, 700, 5000])
@pytest.mark.parametrize("offset", [0.0, 30.0, -100.0, 1e3, 1e5, -1e7, -1497613952.0])
def test_gradient_of_offset_rows(V, offset):
    """As norms: d's rounding (below 4 u times log 2, as most weight has |d| < 16), 2^x within 2 units in the last place
    (4 u) and three products give a probability within 8 u, the factor beside it another 8 u of its terms."""
    g = torch.Generator().manual_seed(V)
    rows = 64
    x = (torch.randn(rows, V, generator=g) * max(2.0, 2e-7 * abs(offset))).double().add(offset).float().cuda()
    ids = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()
    dl, dh = torch.randn(rows, generator=g).cuda(), torch.randn(rows, generator=g).cuda() * 0.3
    got = orc.scores_grad(x, ids, orc.scores(x, ids), dl, dh).double()
    want = _exact_grad(x, ids, dl, dh)
    want_p = want - torch.zeros_like(want).scatter_(1, ids.long()[:, None], dl.double()[:, None])     # without the tokens' ones
    assert float((got - want).norm() / want_p.norm()) <= 16 * ref.U


@pytest.mark.parametrize("io", list(DT))
@pytest.mark.parametrize("V", [1, 7, 300, 9000])
def test_gradient_of_rows_masked_by_the_lowest_value(io, V):
    """An even row: every probability is 1 / V, and the entropy, at its largest, has no slope."""
    x = torch.full((3, V), torch.finfo(DT[io]).min, dtype=DT[io], device="cuda")
    ids = torch.tensor([0, V // 2, V - 1], dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    got = orc.scores_grad(x, ids, orc.scores(x, ids), one, one).double()
    want = torch.full((3, V), -1.0 / V, dtype=torch.float64, device="cuda").scatter_add_(1, ids.long()[:, None], one.double()[:, None])
    want = want.float().double()                # as any fp32 result is, at best
    tol = 48 * ref.U / V + want.abs() * ref.IO_U[io] + ref.IO_TINY[io]
    assert bool(((got - want).abs() <= tol).all())


def test_scores_made_elsewhere_have_an_lse_alone():
    """The gradient then takes that; it takes the rounding's rest again where the buffers are filled once more."""
    x = torch.randn(5, 300, device="cuda")
    even = torch.full((5, 300), torch.finfo(torch.float32).min, device="cuda")
    ids = torch.arange(5, dtype=torch.int32, device="cuda")
    one = torch.ones(5, device="cuda")
    s, t = orc.scores(x, ids), orc.scores(even, ids)
    logp, entropy, lse, top_ids, top_logp = s
    assert lse.shape == (5,) and top_ids is None and top_logp is None
    want = orc.scores_grad(x, ids, s, one)
    bare = [s._replace(lse=lse.clone()), t._replace(lse=t.lse.copy_(lse))]       # no rest; one that is not lse's any more
    orc.rnn_scores(x, ids, lse=torch.empty_like(lse))
    for other in bare:
        assert float((orc.scores_grad(x, ids, other, one) - want).abs().max()) <= 16 * ref.U
    u = orc.scores(even, ids)
    orc.rnn_scores(x, ids, 0, *u)
    assert torch.equal(u.lse, lse) and torch.equal(orc.scores_grad(x, ids, u, one), want)
    pair = torch.empty(2, 5, device="cuda")
    orc.rnn_scores(x, ids, lse=pair)
    assert torch.equal(pair[0], lse) and torch.equal(orc.scores_grad(x, ids, s._replace(lse=pair), one), want)
    with torch.inference_mode():
        v = orc.scores(x, ids)
        assert torch.equal(orc.scores_grad(x, ids, v, one), want)
