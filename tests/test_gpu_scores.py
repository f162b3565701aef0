"""Token scores and their gradient on the GPU against the 64-bit reference:
types, vocabularies from one to several tiles, odd rows and strides, ties,
masked logits, rows of nothing but -inf, NaN and infinities, tokens left out,
the gradient in place, and the refusals of the binding."""
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


def _rows(x, pad):
    """The rows with `pad` elements between them."""
    if not pad:
        return x.cuda()
    w = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    w[:, :x.shape[1]] = x.cuda()
    return w[:, :x.shape[1]]


def _check(got, x, ids, top, finite=True):
    want = ref.scores(x.double(), ids, top)
    V = x.shape[1]
    xd = x.double()
    # lse: the exponentials' arguments and V sums; logp adds the subtraction at the logits' scale
    span = torch.nan_to_num(xd.masked_fill(torch.isinf(xd), 0.0)).abs().amax(1) + 1
    u = ref.U * (16 + min(V, 64) + V // 64)
    bound = u * (1 + 0 * span) + 8 * ref.U * span + ref.U * want["lse"].abs().nan_to_num(0, 0, 0)
    def same(a, b, tol, what):  # noqa: E306
        a, b = a.double().cpu(), b.double()
        odd = ~torch.isfinite(b)
        assert torch.equal(torch.nan_to_num(a[odd], 7.0), torch.nan_to_num(b[odd], 7.0)), what
        ok = (a - b).abs()[~odd] <= tol.expand_as(b)[~odd]
        assert ok.all(), (what, a[~odd][~ok][:3], b[~odd][~ok][:3], tol.expand_as(b)[~odd][~ok][:3])
    same(got.lse, want["lse"], bound, "lse")
    # entropy: sums of p (|log p| <= span + log V) with the same roundings
    same(got.entropy, want["entropy"], bound * (4 + 2 * span + 2 * torch.log(torch.tensor(float(V) + 1))), "entropy")
    if ids is not None:
        same(got.logp, want["logp"], bound, "logp")
    if top:
        assert torch.equal(got.top_ids.cpu(), want["top_ids"])
        same(got.top_logp, want["top_logp"], bound[:, None], "top_logp")
    return want, bound


CASES = [  # rows, vocab, top, io, pad
    (1, 1, 1, "f32", 0), (3, 2, 2, "bf16", 1), (5, 31, 31, "f16", 0), (4, 33, 32, "f32", 3), (2, 255, 5, "bf16", 0),
    (3, 257, 32, "bf16", 7), (2, 1000, 20, "f16", 8), (7, 4097, 8, "f32", 0), (2, 8191, 32, "bf16", 0),
    (1, 20011, 20, "f16", 0), (700, 130, 4, "bf16", 0), (3, 16384, 0, "bf16", 0), (2, 33000, 32, "f32", 4),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("masked", [False, True])
def test_scores_and_gradient(c, masked):
    rows, V, top, io, pad = c
    g = torch.Generator().manual_seed(rows * 1000 + V)
    x = (torch.randn(rows, V, generator=g) * 3).to(DT[io])
    ids = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32)
    if masked:
        x[torch.rand(rows, V, generator=g) < 0.4] = -INF
        x[0] = -INF                                # nothing allowed
        if rows > 2:
            ids[1] = -1
            x[2, :] = -INF
            x[2, V // 2] = 1.5                     # one left
    X = _rows(x, pad)
    got = orc.scores(X, ids.cuda(), top=top)
    want, bound = _check(got, x, ids, top)
    dl, dh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    dt = torch.randn(rows, top, generator=g) if top else None
    mine = orc.scores_grad(X, ids.cuda(), got, dl.cuda(), dh.cuda(), None if dt is None else dt.cuda())
    expect = ref.scores_grad(x.double(), ids, want, dl.double(), dh.double(), None if dt is None else dt.double())
    w = dl.abs() + (0 if dt is None else dt.abs().sum(1))
    p = torch.exp(x.double() - want["lse"][:, None]).nan_to_num(0, 0, 0)
    spread = (x.double() - want["lse"][:, None]).abs().nan_to_num(0, 0, 0) + want["entropy"][:, None].abs()
    rel = 4 * bound[:, None] + 16 * ref.U
    extra = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0).long()[:, None], dl.double().abs()[:, None])
    if dt is not None:
        extra.scatter_add_(1, want["top_ids"].long(), dt.double().abs())
    tol = rel * p * (w.double()[:, None] + dh.double().abs()[:, None] * (spread + 1 + bound[:, None] * 50)) + (top + 4) * ref.U * extra
    ref.close(mine, expect, tol, io, "dlogits")
    # in place: the same bits
    inplace = X.clone() if not pad else _rows(x, pad)
    orc.rnn_scores_grad(inplace, ids.cuda(), got, dl.cuda(), dh.cuda(), None if dt is None else dt.cuda(), dlogits=inplace)
    assert torch.equal(inplace, mine)


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    rows, V, top = 4, 300, 3
    x = torch.randn(rows, V, generator=g)
    ids = torch.tensor([5, 0, -1, 299], dtype=torch.int32)
    dl, dh, dt = (torch.randn(*s, generator=g) for s in ((rows,), (rows,), (rows, top)))
    s = orc.scores(x.cuda(), ids.cuda(), top=top)
    mine = orc.scores_grad(x.cuda(), ids.cuda(), s, dl.cuda(), dh.cuda(), dt.cuda()).cpu().double()

    def f(v):
        o = ref.scores(v, ids, top)
        return float((o["logp"] * dl).sum() + (o["entropy"] * dh).sum() + (o["top_logp"] * dt).sum())
    for _ in range(4):
        way = torch.randn(rows, V, generator=g).double()
        slope = (f(x.double() + 1e-6 * way) - f(x.double() - 1e-6 * way)) / 2e-6
        assert abs(slope - float((mine * way).sum())) <= 1e-4 * float((mine.abs() * way.abs()).sum())


def test_ties_take_the_lowest_place():
    V = 5000
    x = torch.zeros(3, V)
    x[1] = torch.arange(V) % 7
    x[2, ::2] = -0.0                     # +0 and -0 tie
    for io in DT:
        got = orc.scores(x.to(DT[io]).cuda(), top=32)
        assert got.logp is None
        assert torch.equal(got.top_ids[0].cpu(), torch.arange(32, dtype=torch.int32))
        assert torch.equal(got.top_ids[1].cpu(), torch.arange(6, 6 + 7 * 32, 7, dtype=torch.int32))
        assert torch.equal(got.top_ids[2].cpu(), torch.arange(32, dtype=torch.int32))


def test_sorted_rows_either_way():
    V = 9000
    up = torch.arange(V, dtype=torch.float32) / 512
    got = orc.scores(torch.stack([up, up.flip(0)]).cuda(), top=32)
    assert torch.equal(got.top_ids[0].cpu(), torch.arange(V - 1, V - 33, -1, dtype=torch.int32))
    assert torch.equal(got.top_ids[1].cpu(), torch.arange(32, dtype=torch.int32))


@pytest.mark.parametrize("io", list(DT))
def test_nan_and_infinities(io):
    V = 700
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, V, generator=g)
    x[0, 600] = float("nan")
    x[1, 3] = INF
    x[2, 10], x[2, 20] = INF, float("nan")
    x[3, 5:] = -INF
    x[4] = -INF
    x[5] = torch.finfo(DT[io]).min          # a mask by the type's lowest value: an even row
    x = x.to(DT[io])
    ids = torch.tensor([1, 1, 1, 2, 2, V], dtype=torch.int32)      # the last: no such token
    got = orc.scores(x.cuda(), ids.cuda(), top=6)
    want, _ = _check(got, x, ids, 6)
    assert got.logp[5].isnan() and got.top_ids[0, 0] == 600 and got.top_ids[2, :2].tolist() == [20, 10]
    one = torch.ones(6, device="cuda")
    d = orc.scores_grad(x.cuda(), ids.clamp(max=V - 1).cuda(), got, one, one)
    assert d[:3].isnan().all() and not d[4].any()
    assert torch.isfinite(d[3:].float()).all() and not d[3, 5:].any()


def test_rows_far_apart():
    """Rows whose offsets pass 2^31 elements."""
    V, stride = 64, 1 << 30
    if torch.cuda.get_device_properties(0).total_memory < 12 << 30:
        pytest.skip("needs 9 GB")
    whole = torch.empty(4 * stride + V, dtype=torch.float16, device="cuda")
    x = whole.as_strided((5, V), (stride, 1))
    v = torch.randn(5, V, generator=torch.Generator().manual_seed(2)).half()
    x.copy_(v.cuda())
    ids = torch.arange(5, dtype=torch.int32)
    got = orc.scores(x, ids.cuda(), top=5)
    _check(got, v, ids, 5)
    d = orc.scores_grad(x, ids.cuda(), got, torch.ones(5, device="cuda"))
    assert torch.equal(d, orc.scores_grad(v.cuda(), ids.cuda(), got, torch.ones(5, device="cuda")))


def test_no_rows_and_refusals():
    x = torch.zeros(0, 9, device="cuda")
    assert orc.scores(x, torch.zeros(0, dtype=torch.int32, device="cuda"), top=3).top_ids.shape == (0, 3)
    x = torch.zeros(2, 9, device="cuda")
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: orc.scores(x.double(), ids), lambda: orc.scores(x, ids.long()), lambda: orc.scores(x.t(), ids),
                lambda: orc.scores(x, ids[:1]), lambda: orc.scores(x.cpu(), ids), lambda: orc.scores(x, ids, top=-1)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for top in (10, 33):
        with pytest.raises(orc.RNNError) as e:
            orc.scores(x, ids, top=top)
        assert e.value.status == 1
    s = orc.scores(x, ids)
    with pytest.raises(orc.RNNError):
        orc.scores_grad(x, None, s, torch.ones(2, device="cuda"))
    with pytest.raises(orc.RNNError):
        orc.rnn_scores_grad(x, ids, s._replace(lse=None), torch.ones(2, device="cuda"), dlogits=torch.empty_like(x))


@pytest.mark.parametrize("rows,V", [(2, 3000), (3, 50001), (700, 9000)])
def test_many_equal_logits(rows, V):
    """Rows in which hundreds of logits tie at the last place wanted, with larger ones among and after them."""
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-3, 4, (rows, V), generator=g).float()       # seven values: a seventh of the row ties at the top
    x[0] = -INF
    x[0, V - 7:V - 2] = torch.arange(5).float()                    # five allowed, at the row's end; the rest tie at -inf
    x[1, torch.randperm(V, generator=g)[:900]] = torch.rand(900, generator=g) + 10.0
    for io in ("bf16", "f32"):
        v = x.to(DT[io])
        got = orc.scores(v.cuda(), top=32)
        assert torch.equal(got.top_ids[:3].cpu(), ref.scores(v[:3].double(), None, 32)["top_ids"])
