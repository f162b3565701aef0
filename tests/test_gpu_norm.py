"""Layer normalisation on the GPU against its formula in 64 bits.

Bounds: with z and w = dY W of a row of D values, sums err by at most D u of their absolute terms (in
norm by sqrt(D) u, which is not needed here), a handful of operations by 8 u: Y by (D + 8) u
(|z W| + |bias|) + D u |W| (the mean's error, relative to the deviation, times rstd: at most D u max|x| rstd);
dX by rstd (2 D + 8) u (|w| + mean|w| + |z| mean|w z|); column sums of R rows by (R + D + 8) u of their absolute terms."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def _within(got, want, bound, io, what):
    got = got.double().cpu()
    tol = bound + (want.abs() + bound) * ref.IO_U[io] + ref.IO_TINY[io]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}"


def _check(X, W, bias, dY, io, plan, eps, stride=0):
    D, R = X.shape[-1], X.numel() // X.shape[-1]
    Y, stats = orc.layer_norm(plan, X, W, bias)
    out = orc.layer_norm_grad(plan, dY, X, stats, W, bias)
    up = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    x, w_, b_, dy = up(X).reshape(R, D), up(W), up(bias), up(dY).reshape(R, D)
    y, mean, rstd = ref.norm(x, w_, b_, eps)
    wide = torch.ones(D, dtype=torch.float64) if w_ is None else w_
    z = (x - mean[:, None]) * rstd[:, None]
    off = D * U * x.abs().amax(1, keepdim=True) * rstd[:, None]       # z's error: the mean's, rstd's and its own
    ez = off + (D + 8) * U * z.abs()
    _within(Y.reshape(R, D), y, ez * wide.abs() + 4 * U * y.abs() + 2 * U * (0 if b_ is None else b_.abs()), io, "Y")
    _within(stats[:, 0], mean, D * U * x.abs().mean(1), "f32", "mean")
    _within(stats[:, 1], rstd, (D + 8) * U * rstd + off[:, 0] ** 2 * rstd, "f32", "rstd")
    w = dy * wide
    m1, m2 = w.mean(1, keepdim=True), (w * z).mean(1, keepdim=True)
    want = rstd[:, None] * (w - m1 - z * m2)
    size = w.abs() + w.abs().mean(1, keepdim=True) + z.abs() * (w * z).abs().mean(1, keepdim=True)
    bound = rstd[:, None] * ((2 * D + 16) * U * size + ez * m2.abs() + z.abs() * (w.abs() * ez).mean(1, keepdim=True))
    _within(out["dX"].reshape(R, D), want, bound, io, "dX")
    if w_ is not None:
        _within(out["dW"], (dy * z).sum(0), (R + 8) * U * (dy * z).abs().sum(0) + (dy.abs() * ez).sum(0), "f32", "dW")
    if b_ is not None:
        _within(out["dbias"], dy.sum(0), R * U * dy.abs().sum(0), "f32", "dbias")
    return Y, stats, out


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 64), (2, 129), (70, 257), (33, 1001), (4, 2048), (1, 3001), (3, 8192),
                                   (2, 12345), (2, 32768), (300, 40)], ids=str)
def test_rows(shape, io):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    R, D = shape
    plan = orc.rnn_norm_create(D, eps=1e-5)
    orc.rnn_norm_set_io_type(plan, io)
    X, dY = (r(R, D) * 2 + 1).to(DT[io]).cuda(), r(R, D).to(DT[io]).cuda()
    _check(X, (1 + 0.3 * r(D)).cuda(), r(D).cuda(), dY, io, plan, 1e-5)
    _check(X, None, None, dY, io, plan, 1e-5)


def test_rows_far_from_zero():
    g = torch.Generator().manual_seed(2)
    plan = orc.rnn_norm_create(500, eps=1e-6)
    X, dY = (torch.randn(9, 500, generator=g) + 1000.0).cuda(), torch.randn(9, 500, generator=g).cuda()
    _check(X, None, None, dY, "f32", plan, 1e-6)


def test_constant_rows_and_rows_with_nan():
    plan = orc.rnn_norm_create(48, eps=1e-5)
    X = torch.randn(4, 48, device="cuda")
    X[0], X[1, 5], X[2, 7] = 3.0, float("nan"), float("inf")
    b = torch.randn(48, device="cuda")
    Y, stats = orc.layer_norm(plan, X, None, b)
    assert torch.equal(Y[0], b) and Y[1].isnan().all() and Y[2].isnan().all() and Y[3].isfinite().all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_parts_of_wider_rows(io, off):
    g = torch.Generator().manual_seed(3)
    D = 96
    plan = orc.rnn_norm_create(D)
    orc.rnn_norm_set_io_type(plan, io)
    big, dbig = (torch.randn(2, 7, 3 * D + 8, generator=g).to(DT[io]).cuda() for _ in range(2))
    X, dY = big[..., D + off:2 * D + off], dbig[..., off:D + off]
    W = torch.randn(D, generator=g).cuda()
    Y, stats, out = _check(X, W, None, dY, io, plan, 1e-5)
    keep = big.clone()
    orc.rnn_layer_norm(plan, X, W, None, X)                 # in place
    assert torch.equal(X, Y)
    keep[..., D + off:2 * D + off] = Y
    assert torch.equal(big, keep)


@pytest.mark.parametrize("D", [96, 4096])
def test_gradient_in_place_and_alone(D):
    g = torch.Generator().manual_seed(4)
    plan = orc.rnn_norm_create(D)
    X, dY, W = (torch.randn(*s, generator=g).cuda() for s in ((50, D), (50, D), (D,)))
    _, stats = orc.layer_norm(plan, X, W, W)
    full = orc.layer_norm_grad(plan, dY, X, stats, W, W)
    for name, t in full.items():
        one = torch.empty_like(t)
        orc.rnn_layer_norm_grad(plan, dY, X, stats, W, **{name: one})
        assert torch.equal(one, t), name
    for which in (0, 1):
        a, b = dY.clone(), X.clone()
        dW, dbias = torch.empty_like(W), torch.empty_like(W)
        orc.rnn_layer_norm_grad(plan, a, b, stats, W, (a, b)[which], dW, dbias)
        assert torch.equal((a, b)[which], full["dX"]) and torch.equal(dW, full["dW"]) and torch.equal(dbias, full["dbias"])


def test_no_rows():
    plan = orc.rnn_norm_create(8)
    X, W = torch.empty(0, 8, device="cuda"), torch.ones(8, device="cuda")
    Y, stats = orc.layer_norm(plan, X, W, W)
    assert Y.shape == (0, 8) and stats.shape == (0, 2)
    out = orc.layer_norm_grad(plan, Y, X, stats, W, W)
    assert not out["dW"].any() and not out["dbias"].any()


def test_captured_and_on_another_stream():
    g = torch.Generator().manual_seed(5)
    X, dY, W = (torch.randn(*s, generator=g).cuda() for s in ((200, 512), (200, 512), (512,)))
    ready = orc.rnn_norm_create(512)
    Y, stats = orc.layer_norm(ready, X, W, W)
    want = orc.layer_norm_grad(ready, dY, X, stats, W, W)
    plan = orc.rnn_norm_create(512)
    y, s2, out = torch.empty_like(Y), torch.empty_like(stats), {n: torch.empty_like(t) for n, t in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orc.rnn_layer_norm(plan, X, W, W, y, s2)
        orc.rnn_layer_norm_grad(plan, dY, X, s2, W, **out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, Y) and all(torch.equal(out[n], want[n]) for n in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y2, st2 = orc.layer_norm(plan, X, W, W, stream=side)
    out2 = orc.layer_norm_grad(plan, dY, X, st2, W, W, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(Y2, Y) and all(torch.equal(out2[n], want[n]) for n in want)
