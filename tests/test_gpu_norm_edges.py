"""Layer normalisation of rows far from zero, and of so many rows that blocks walk them, against its formula in 64 bits.

Bounds.  A thread adds at most 32 values, a warp five times, a row's warps at most 32 times: sums of a row err by at most P = 72 u
of their absolute terms, their quotients by D by one more u.  So the mean is off by c of at most (P + 1) u max|x|, d = x - mean by u |d|, and the
mean of d, which is taken off it, by (P + 1) u mean|d|: with m = mean|d|, z is off by
    ez = rstd ((P + 2) u m + 2 u |d|) + |z| er,
where er, of rstd, is ((P + 4) u (mean d^2 + c^2)) rstd^2 / 2 + 4 u.  |d| is at most that of the exact mean and |c|."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
P = 72


def _within(got, want, bound, io, what):
    got = got.double()
    tol = bound + (want.abs() + bound) * ref.IO_U[io] + ref.IO_TINY[io]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}, " \
                          f"off by {float(((got - want).abs() / tol).max()):.2f} of what it may be"


def _check(X, W, bias, dY, io, eps):
    R, D = X.shape
    plan = orc.rnn_norm_create(D, eps=eps)
    orc.rnn_norm_set_io_type(plan, io)
    Y, stats = orc.layer_norm(plan, X, W, bias)
    out = orc.layer_norm_grad(plan, dY, X, stats, W, bias)
    x, w, b, dy = (t.double() for t in (X, W, bias, dY))
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    z = (x - mean) * rstd
    c = (P + 1) * U * x.abs().amax(1, keepdim=True)
    d = (x - mean).abs() + c
    er = (P + 4) * U * ((d * d).mean(1, keepdim=True) + c * c) * rstd ** 2 / 2 + 4 * U
    ez = rstd * ((P + 2) * U * d.mean(1, keepdim=True) + 2 * U * d) + z.abs() * er
    y = z * w + b
    _within(Y, y, ez * w.abs() + 4 * U * (y.abs() + b.abs()), io, "Y")
    # (held as one fp32 number)
    _within(stats[:, :1], mean, (P + 1) * U * d.mean(1, keepdim=True) + U * mean.abs(), "f32", "mean")
    _within(stats[:, 1:], rstd, er * rstd, "f32", "rstd")
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * z).mean(1, keepdim=True)
    # v is formed of sums over d, c among it
    far = (g.abs() * d).mean(1, keepdim=True) * rstd
    size = g.abs() + g.abs().mean(1, keepdim=True) + z.abs() * far
    bound = rstd * ((2 * P + 16) * U * size + ez * m2.abs() + z.abs() * (g.abs() * ez).mean(1, keepdim=True) + er * size)
    _within(out["dX"], rstd * (g - m1 - z * m2), bound, io, "dX")
    # a row's value and its term are rounded; sums over rows: a thread's rows, its parts' 16 threads, in turn
    _within(out["dW"], (dy * z).sum(0), (R + 8) * U * (dy * z).abs().sum(0) + (dy.abs() * ez).sum(0), "f32", "dW")
    _within(out["dbias"], dy.sum(0), (R + 8) * U * dy.abs().sum(0), "f32", "dbias")


def _inputs(R, D, io, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(R, D).to(DT[io]), 1 + 0.3 * r(D), r(D), r(R, D).to(DT[io])


@pytest.mark.parametrize("shape", [(9, 500), (5, 48), (70, 257), (7, 2048), (3, 5000), (3, 12345), (2600, 300), (2600, 2048)], ids=str)
@pytest.mark.parametrize("far", [1000.0, -1e4, 1e6])
def test_rows_far_from_zero(shape, far):
    X, W, b, dY = _inputs(*shape, "f32")
    _check(X + far, W, b, dY, "f32", 1e-6)


@pytest.mark.parametrize("rows,D", [(3, D) for D in (1, 48, 768, 1001, 2048, 8192, 12345)] + [(2600, D) for D in (1, 48, 768, 1001, 2048)])
def test_constant_rows(rows, D):
    """Every d is the same: what is left of it after their mean is at most (P + 2) u of c, (P + 1) u |x|."""
    W, b = torch.full((D,), 1.5, device="cuda"), torch.linspace(-1, 1, D, device="cuda")
    X = torch.empty(rows, D, device="cuda")
    X[0::3], X[1::3], X[2::3] = 1000.1, 0.1, -33333.3
    for eps in (1e-5, 1e-12):
        plan = orc.rnn_norm_create(D, eps=eps)
        Y, stats = orc.layer_norm(plan, X, W, b)
        bound = (P + 2) * (P + 1) * U * U * X.abs().double() * eps ** -0.5 * 1.5 + 4 * U
        assert ((Y.double() - b.double()).abs() <= bound).all(), float((Y - b).abs().max())
        assert torch.equal(stats[:, 0], X[:, 0])
        dY = torch.randn(rows, D, device="cuda")
        out = orc.layer_norm_grad(plan, dY, X, stats, W, b)
        assert float(out["dW"].abs().max()) <= float((dY.abs().double() * bound).sum(0).max())


# from 16 rows a multiprocessor on, blocks walk rows with 32 values a thread: a shape for each range of sizes, of whole pieces of 16
# bytes and not
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [264, 1001, 1024, 1025, 2048, 3001, 4096, 5003, 8192, 8200, 9001])
def test_many_rows(D, io):
    rows = 16 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    X, W, b, dY = _inputs(rows, D, io, seed=D)
    _check((2 * X.float() + 1).to(DT[io]), W, b, dY, io, 1e-5)


def test_many_rows_in_place_and_of_wider_rows():
    rows, D = 16 * torch.cuda.get_device_properties(0).multi_processor_count + 5, 520
    for off in (0, 1):
        big = torch.randn(rows, 3 * D, device="cuda")
        X = big[:, D + off:2 * D + off]
        plan = orc.rnn_norm_create(D)
        keep = big.clone()
        want, _ = orc.layer_norm(plan, X.contiguous(), None, None)
        orc.rnn_layer_norm(plan, X, None, None, X)
        # (rows off a boundary are added in another order: a few units of the largest value)
        assert ((X - want).abs() <= 200 * U * (1 + want.abs())).all()
        keep[:, D + off:2 * D + off] = X
        assert torch.equal(big, keep)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [96, 8200])
def test_inputs_whose_rows_are_one(D, io):
    X, W, b, dY = _inputs(1, D, io)
    plan = orc.rnn_norm_create(D)
    orc.rnn_norm_set_io_type(plan, io)
    many = X.expand(50, D)
    want, stats = orc.layer_norm(plan, many.contiguous(), W, b)
    Y, st = orc.layer_norm(plan, many, W, b)
    assert torch.equal(Y, want) and torch.equal(st, stats)
    slopes = dY.expand(5, 10, D)
    full = orc.layer_norm_grad(plan, slopes.reshape(50, D).contiguous(), many.contiguous(), stats, W, b)
    out = orc.layer_norm_grad(plan, slopes, X.expand(5, 10, D), stats, W, b)
    for name in full:
        assert torch.equal(out[name].view_as(full[name]), full[name]), name
    with pytest.raises(ValueError):
        orc.rnn_layer_norm(plan, many, W, b, many)


@pytest.mark.parametrize("rows", [3, 2600])
def test_constant_rows_whose_error_has_no_square(rows):
    """The mean of values of 10^30 may be off by more than the root of the largest number: no NaN comes of that."""
    D = 768
    plan = orc.rnn_norm_create(D)
    X, b = torch.linspace(1.1e29, 1.1e30, rows, device="cuda")[:, None].repeat(1, D), torch.randn(D, device="cuda")
    Y, _ = orc.layer_norm(plan, X, None, b)
    assert torch.equal(Y, b.expand(rows, D))
