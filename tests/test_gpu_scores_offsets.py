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
