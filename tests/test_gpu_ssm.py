"""State space operators on the GPU against the 64-bit references: types,
layouts, lengths from zero to several tiles, odd channels, groups and state
sizes, carried states, views into wider tensors, rows with nothing in them,
single tokens with slots, gradients against the formulas and against
differences, other streams, and the refusals the binding and kernels make."""
import pytest
import torch

import onnx_recurrent_gb300 as orc
import ssm_ref64 as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    orc.build()


def _gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0: torch.randn(*s, generator=g) * scale


def _lens(kind, N, S):
    if kind is None:
        return None
    base = [S, 0, 1, max(0, S - 1), S // 2, min(S, 16), min(S, 17), min(S, 15)]
    return torch.tensor([base[i % len(base)] for i in range(N)], dtype=torch.int32)


def _lead(t, layout):
    """[N, S, ...] data as the layout's tensor."""
    return t if layout == 1 else t.transpose(0, 1).contiguous()


def _wide_view(t, pad_before, pad_after):
    """The same values as the middle part of a wider last dimension, NaN around them."""
    shape = t.shape[:-1] + (t.shape[-1] + pad_before + pad_after,)
    w = torch.full(shape, float("nan"), dtype=t.dtype, device=t.device)
    v = w[..., pad_before:pad_before + t.shape[-1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------ convolution

CONV = [  # N, S, D, K, io, layout, lens, carried, act, bias, view
    (1, 1, 1, 4, "f32", 0, None, False, "silu", True, False),
    (2, 5, 7, 1, "f32", 1, None, False, "silu", True, False),
    (3, 33, 130, 2, "bf16", 1, True, True, "silu", True, False),
    (8, 64, 64, 3, "f16", 0, True, True, None, True, False),
    (5, 70, 257, 4, "f32", 1, True, True, "silu", False, True),
    (2, 129, 512, 4, "bf16", 0, None, False, "silu", True, False),
    (2, 100, 96, 4, "bf16", 1, True, False, "silu", True, True),
    (3, 40, 24, 8, "f32", 0, True, True, "silu", True, False),
    (2, 37, 40, 5, "f16", 1, None, True, None, True, False),
    (8, 3, 128, 4, "f32", 1, True, True, "silu", True, False),     # steps fewer than taps
    (4, 300, 1024, 4, "bf16", 1, True, True, "silu", True, False),
]


def _conv_case(c, seed=0):
    N, S, D, K, io, layout, lens, carried, act, bias, view = c
    r = _gen(seed)
    x, W = r(N, S, D).to(DT[io]), r(D, K, scale=0.5)
    b = r(D, scale=0.3) if bias else None
    h0 = r(N, K - 1, D).to(DT[io]) if carried else None
    dY, dhT = r(N, S, D).to(DT[io]), r(N, K - 1, D).to(DT[io])
    return x, W, b, h0, dY, dhT, _lens(lens, N, S)


def _d(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("c", CONV, ids=lambda c: "-".join(map(str, c)))
def test_conv_and_gradient(c):
    N, S, D, K, io, layout, lens, carried, act, bias, view = c
    x, W, b, h0, dY, dhT, ln = _conv_case(c)
    plan = orc.rnn_ssm_create(D, conv_width=K, layout=layout, activation=act)
    orc.rnn_ssm_set_io_type(plan, io)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    X, DY = _lead(x, layout).cuda(), _lead(dY, layout).cuda()
    if view:
        X, DY = _wide_view(X, 8, 3), _wide_view(DY, 1, 0)
    Y, state = orc.ssm_conv(plan, X, cu(W), cu(b), cu(ln), cu(h0))
    rY, rT, pre = ref.conv(_d(x), _d(W), _d(b), ln, _d(h0), act == "silu")
    hist = torch.zeros(N, K - 1, D, dtype=torch.float64) if h0 is None else _d(h0).abs()
    mag = torch.zeros(N, S, D, dtype=torch.float64) + (0 if b is None else b.double().abs())
    line = torch.cat([hist, x.double().abs()], 1)
    for k in range(K):
        mag = mag + line[:, k:k + S] * W.double()[:, k].abs()
    # K products and sums, silu (slope at most 1.1) with its own 8 roundings
    bound = (1.1 * (2 * K + 2) + 8) * ref.U * mag
    back = (lambda t: t) if layout == 1 else (lambda t: t.transpose(0, 1))
    ref.close(back(Y), rY, bound, io, "Y")
    assert torch.equal(state.cpu().double(), rT)
    g = orc.ssm_conv_grad(plan, DY, X, cu(W), cu(b), cu(ln), cu(h0), cu(dhT))
    args = (_d(dY), _d(dhT), _d(x), _d(W), _d(b), ln, _d(h0), act == "silu")
    want, mags = ref.conv_grad(*args), ref.conv_grad(*args, magnitude=True)
    u = ref.U * (4 * K + 40)
    ref.close(back(g["dX"]), want["dX"], u * mags["dX"], io, "dX")
    ref.close(g["dW"], want["dW"], (u + N * S * ref.U) * mags["dW"], "f32", "dW")
    if bias:
        ref.close(g["dbias"], want["dbias"], (u + N * S * ref.U) * mags["dbias"], "f32", "dbias")
    if carried:
        ref.close(g["d_initial_state"], want["d_initial_state"], u * mags["d_initial_state"], io, "d_initial_state")
    orc.rnn_ssm_sync(plan)


def test_conv_in_pieces_is_the_whole():
    """A prompt taken in pieces, the state carried, then token by token: bit for bit the whole prompt's outputs."""
    r = _gen(5)
    N, S, D, K = 3, 50, 72, 4
    x, W, b = r(N, S, D).bfloat16().cuda(), r(D, K).cuda(), r(D).cuda()
    plan = orc.rnn_ssm_create(D, conv_width=K, layout=1)
    orc.rnn_ssm_set_io_type(plan, "bf16")
    Y, last = orc.ssm_conv(plan, x, W, b)
    state, parts = None, []
    for lo, hi in ((0, 1), (1, 3), (3, 35), (35, 44)):
        y, state = orc.ssm_conv(plan, x[:, lo:hi], W, b, None, state)
        parts.append(y)
    for t in range(44, S):
        y = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
        orc.rnn_ssm_conv_step(plan, x[:, t], W, b, state, y)
        parts.append(y[:, None])
    assert torch.equal(torch.cat(parts, 1), Y) and torch.equal(state, last)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,D,K", [(1, 5, 4), (7, 264, 2), (3, 1000, 8), (64, 129, 3), (2, 6, 1)])
def test_conv_step(io, N, D, K):
    r = _gen(6)
    x, st, W, b = r(N, D).to(DT[io]), r(N, K - 1, D).to(DT[io]), r(D, K), r(D)
    plan = orc.rnn_ssm_create(D, conv_width=K)
    orc.rnn_ssm_set_io_type(plan, io)
    X = _wide_view(x.cuda(), 3, 2)
    Y, out = torch.empty(N, D, dtype=DT[io], device="cuda"), torch.full((N, K - 1, D), 9.0, dtype=DT[io], device="cuda")
    state = st.cuda()
    orc.rnn_ssm_conv_step(plan, X, W.cuda(), b.cuda(), state, Y, state_out=out)
    rY, rT, _ = ref.conv(x.double()[:, None], W.double(), b.double(), None, st.double(), True)
    mag = b.double().abs() + (torch.cat([st, x[:, None]], 1).double().abs() * W.double().abs().T).sum(1)
    ref.close(Y, rY[:, 0], (1.1 * (2 * K + 2) + 8) * ref.U * mag, io, "Y")
    assert torch.equal(out.cpu().double(), rT) and torch.equal(state.cpu(), st)
    # slots: a permutation with padding; untouched slots keep their values
    if N >= 3:
        cache = torch.full((N + 4, K - 1, D), 5.0, dtype=DT[io], device="cuda")
        slots = torch.randperm(N + 4, generator=torch.Generator().manual_seed(1))[:N].int()
        cache[slots.long().cuda()] = st.cuda()
        slots[1] = -1
        Y2 = torch.empty_like(Y)
        orc.rnn_ssm_conv_step(plan, X, W.cuda(), b.cuda(), cache, Y2, slots=slots.cuda())
        keep = torch.ones(N, dtype=torch.bool)
        keep[1] = False
        assert torch.equal(Y2[keep.cuda()], Y[keep.cuda()]) and not Y2[1].any()
        assert torch.equal(cache[slots[keep].long().cuda()], out[keep.cuda()])
        orc.rnn_ssm_sync(plan)
        slots[0] = N + 4
        orc.rnn_ssm_conv_step(plan, X, W.cuda(), b.cuda(), cache, Y2, slots=slots.cuda())
        with pytest.raises(orc.RNNError) as e:
            orc.rnn_ssm_sync(plan)
        assert e.value.status == 2
        orc.rnn_ssm_sync(plan)


# ------------------------------------------------------------ scan

SCAN = [  # N, S, D, M, G, io, layout, lens, carried, gate, skip, soft
    (1, 1, 1, 1, 1, "f32", 1, None, False, True, True, True),
    (2, 1, 40, 16, 1, "bf16", 0, None, True, True, True, True),
    (8, 35, 37, 16, 1, "f32", 1, True, True, True, True, True),
    (8, 48, 64, 16, 2, "bf16", 0, True, True, True, True, True),
    (3, 33, 66, 12, 3, "f32", 0, True, False, False, True, True),
    (2, 20, 10, 5, 2, "f16", 1, None, True, True, False, True),
    (2, 31, 24, 33, 1, "f32", 1, True, True, True, True, False),
    (2, 17, 20, 64, 4, "bf16", 1, None, False, True, True, True),
    (1, 18, 9, 128, 1, "f32", 0, None, True, True, True, True),
    (2, 16, 130, 4, 1, "f16", 1, True, True, False, False, True),
    (1, 150, 136, 16, 1, "f32", 1, None, False, True, True, True),
    (1, 260, 256, 16, 1, "bf16", 1, None, True, True, True, True),
    (2, 67, 260, 8, 2, "f32", 0, True, True, True, True, True),
    (1, 1100, 32, 16, 1, "f32", 1, None, True, True, True, True),     # long enough to be split over time
    (2, 700, 40, 2, 1, "bf16", 0, True, True, True, True, True),
]


def _scan_case(c, seed=0):
    N, S, D, M, G, io, layout, lens, carried, gate, skip, soft = c
    r = _gen(seed)
    t = DT[io]
    v = dict(X=r(N, S, D).to(t), dt=r(N, S, D, scale=0.5).to(t),
             A=-torch.exp(r(D, M, scale=0.7)), B=r(N, S, G, M).to(t), C=r(N, S, G, M).to(t),
             D=r(D) if skip else None, Z=r(N, S, D).to(t) if gate else None,
             dt_bias=r(D, scale=0.5) - 2.0, h0=r(N, D, M) if carried else None)
    if not soft:        # the step itself: small and positive in the main, as the formulas need no sign
        v["dt"] = (v["dt"].float() * 0.1 + 0.05).to(t)
        v["dt_bias"] = None
    return v, r(N, S, D).to(t), r(N, D, M), _lens(lens, N, S)


def _scan_run(c, v, dY, dYh, ln, views=False, stream=None):
    N, S, D, M, G, io, layout, lens, carried, gate, skip, soft = c
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=layout, softplus=soft)
    orc.rnn_ssm_set_io_type(plan, io)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    seq = lambda t: None if t is None else _lead(t, layout).cuda()  # noqa: E731
    X, dt, Z, DY, B, C = seq(v["X"]), seq(v["dt"]), seq(v["Z"]), seq(dY), seq(v["B"]), seq(v["C"])
    if views:
        X, dt, DY = _wide_view(X, 8, 8), _wide_view(dt, 0, 5), _wide_view(DY, 3, 1)
        Z = None if Z is None else _wide_view(Z, 16, 0)
        bc = torch.full(B.shape[:2] + (3, G, M), float("nan"), dtype=B.dtype, device="cuda")
        bc[:, :, 0], bc[:, :, 2] = B, C
        B, C = bc[:, :, 0], bc[:, :, 2]
    args = (X, dt, cu(v["A"]), B, C, cu(v["D"]), Z, cu(v["dt_bias"]), cu(ln), cu(v["h0"]))
    Y, Yh, saved = orc.ssm_scan(plan, *args, save=True, stream=stream)
    g = orc.ssm_scan_grad(plan, DY, saved, *args, dY_h=cu(dYh), stream=stream)
    Y2, Yh2, none = orc.ssm_scan(plan, *args, stream=stream)      # without saving
    torch.cuda.synchronize()
    # a NaN equals nothing, itself least of all
    assert none is None and torch.equal(Y2.nan_to_num(77.0), Y.nan_to_num(77.0)) and torch.equal(Yh2.nan_to_num(77.0), Yh.nan_to_num(77.0))
    orc.rnn_ssm_sync(plan)
    back = (lambda t: t) if layout == 1 else (lambda t: t.transpose(0, 1))
    out = {"Y": back(Y), "Y_h": Yh}
    for k, t in g.items():
        out[k] = back(t) if k in ("dX", "ddt", "dB", "dC", "dZ") else t
    return out


def _check_scan(c, v, dY, dYh, ln, got):
    N, S, D, M, G, io, layout, lens, carried, gate, skip, soft = c
    d = {k: _d(t) for k, t in v.items()}
    a = (d["X"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["Z"], d["dt_bias"], ln, d["h0"], soft)
    rY, rYh, _, _, delta, _ = ref.scan(*a)
    mY, mYh = ref.scan(*a, magnitude=True)[:2]
    rate = float((delta[..., None] * d["A"].abs()).max())
    u = ref.steps_bound(S, M, rate)
    ref.close(got["Y"], rY, u * mY, io, "Y")
    ref.close(got["Y_h"], rYh, u * mYh, "f32", "Y_h")
    want, mags = ref.scan_grad(_d(dY), _d(dYh), *a), ref.scan_grad(_d(dY), _d(dYh), *a, magnitude=True)
    for k, t in got.items():
        if k in ("Y", "Y_h"):
            continue
        terms = {"dB": D // G, "dC": D // G, "dA": N * S, "dD": N * S, "ddt_bias": N * S}.get(k, M)
        w = 2 * ref.steps_bound(S, terms, rate)       # the state and the slope each pass S steps
        ref.close(t, want[k], w * mags[k], "f32" if k in ("dA", "dD", "ddt_bias", "d_initial_h") else io, k)


@pytest.mark.parametrize("c", SCAN, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("views", [False, True])
def test_scan_and_gradient(c, views):
    v, dY, dYh, ln = _scan_case(c)
    _check_scan(c, v, dY, dYh, ln, _scan_run(c, v, dY, dYh, ln, views))


def test_scan_gradient_against_differences():
    """Directional derivatives of the 64-bit forward formulas against the GPU's gradients."""
    c = (2, 25, 20, 7, 2, "f32", 1, True, True, True, True, True)
    v, dY, dYh, ln = _scan_case(c, seed=9)
    got = _scan_run(c, v, dY, dYh, ln)
    names = dict(X="dX", dt="ddt", A="dA", B="dB", C="dC", D="dD", Z="dZ", dt_bias="ddt_bias", h0="d_initial_h")
    d = {k: _d(t) for k, t in v.items()}
    r = _gen(10)

    def loss(w):
        Y, Yh = ref.scan(w["X"], w["dt"], w["A"], w["B"], w["C"], w["D"], w["Z"], w["dt_bias"], ln, w["h0"])[:2]
        return (Y * _d(dY)).sum() + (Yh * _d(dYh)).sum()
    for k, gname in names.items():
        way = r(*d[k].shape).double()
        eps = 1e-6
        up, down = dict(d), dict(d)
        up[k], down[k] = d[k] + eps * way, d[k] - eps * way
        slope = float(loss(up) - loss(down)) / (2 * eps)
        mine = float((got[gname].double().cpu() * way).sum())
        scale = float((got[gname].double().cpu().abs() * way.abs()).sum())
        assert abs(slope - mine) <= 1e-4 * scale + 1e-6, (k, slope, mine)


def test_scan_gradient_bits_repeat():
    c = (4, 90, 200, 16, 1, "bf16", 1, True, True, True, True, True)
    v, dY, dYh, ln = _scan_case(c)
    one, two = _scan_run(c, v, dY, dYh, ln), _scan_run(c, v, dY, dYh, ln)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_scan_in_pieces_and_token_by_token():
    """Carrying the state over pieces and single tokens gives the whole run's outputs (within the bound)."""
    c = (3, 60, 48, 16, 2, "f32", 1, None, False, True, True, True)
    v, _, _, _ = _scan_case(c, seed=4)
    N, S, D, M, G = c[:5]
    cu = {k: None if t is None else t.cuda() for k, t in v.items()}
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G, layout=1)
    h, parts = None, []
    for lo, hi in ((0, 1), (1, 20), (20, 52)):
        p = lambda k: cu[k][:, lo:hi]  # noqa: E731
        y, h, _ = orc.ssm_scan(plan, p("X"), p("dt"), cu["A"], p("B"), p("C"), cu["D"], p("Z"), cu["dt_bias"], None, h)
        parts.append(y)
    for t in range(52, S):
        y = torch.empty(N, D, device="cuda")
        p = lambda k: cu[k][:, t]  # noqa: E731
        orc.rnn_ssm_scan_step(plan, p("X"), p("dt"), cu["A"], p("B"), p("C"), h, y, cu["D"], p("Z"), cu["dt_bias"])
        parts.append(y[:, None])
    d = {k: _d(t) for k, t in v.items()}
    a = (d["X"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["Z"], d["dt_bias"], None, None)
    rY, rYh, _, _, delta, _ = ref.scan(*a)
    mY, mYh = ref.scan(*a, magnitude=True)[:2]
    u = ref.steps_bound(S, M, float((delta[..., None] * d["A"].abs()).max()))
    ref.close(torch.cat(parts, 1), rY, u * mY, "f32", "Y")
    ref.close(h, rYh, u * mYh, "f32", "H")


@pytest.mark.parametrize("N,D,M,G,io", [(1, 1, 1, 1, "f32"), (1, 300, 16, 1, "bf16"), (5, 66, 12, 3, "f16"),
                                        (3, 40, 64, 4, "f32"), (70, 36, 8, 2, "bf16"), (2, 9, 128, 1, "f32"),
                                        (4, 1024, 16, 1, "bf16"), (3, 24, 33, 1, "f32")])
def test_scan_step(N, D, M, G, io):
    c = (N, 1, D, M, G, io, 1, None, True, True, True, True)
    v, _, _, _ = _scan_case(c, seed=2)
    cu = {k: t.cuda() for k, t in v.items()}
    plan = orc.rnn_ssm_create(D, state_size=M, groups=G)
    orc.rnn_ssm_set_io_type(plan, io)
    bc = torch.cat([cu["B"][:, 0].reshape(N, 1, G, M), cu["C"][:, 0].reshape(N, 1, G, M)], 1)
    X, Z = _wide_view(cu["X"][:, 0], 8, 0), _wide_view(cu["Z"][:, 0], 0, 1)
    Y, out = torch.empty(N, D, dtype=DT[io], device="cuda"), torch.empty(N, D, M, device="cuda")
    rest = (cu["D"], Z, cu["dt_bias"])
    orc.rnn_ssm_scan_step(plan, X, cu["dt"][:, 0], cu["A"], bc[:, 0], bc[:, 1], cu["h0"], Y, *rest, H_out=out)
    d = {k: _d(t) for k, t in v.items()}
    a = (d["X"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["Z"], d["dt_bias"], None, d["h0"])
    rY, rH, _, _, delta, _ = ref.scan(*a)
    mY, mH = ref.scan(*a, magnitude=True)[:2]
    u = ref.steps_bound(1, M, float((delta[..., None] * d["A"].abs()).max()))
    ref.close(Y, rY[:, 0], u * mY[:, 0], io, "Y")
    ref.close(out, rH, u * mH, "f32", "H")
    assert torch.equal(cu["h0"].cpu(), v["h0"])
    if N >= 3:
        cache = torch.full((N + 3, D, M), 7.0, device="cuda")
        slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(3))[:N].int()
        cache[slots.long().cuda()] = cu["h0"]
        slots[2] = -1
        Y2 = torch.empty_like(Y)
        orc.rnn_ssm_scan_step(plan, X, cu["dt"][:, 0], cu["A"], bc[:, 0], bc[:, 1], cache, Y2, *rest, slots=slots.cuda())
        keep = torch.ones(N, dtype=torch.bool, device="cuda")
        keep[2] = False
        assert torch.equal(Y2[keep], Y[keep]) and not Y2[2].any()
        assert torch.equal(cache[slots.cuda()[keep].long()], out[keep])
        orc.rnn_ssm_sync(plan)
        slots[0] = N + 3
        orc.rnn_ssm_scan_step(plan, X, cu["dt"][:, 0], cu["A"], bc[:, 0], bc[:, 1], cache, Y2, *rest, slots=slots.cuda())
        with pytest.raises(orc.RNNError) as e:
            orc.rnn_ssm_sync(plan)
        assert e.value.status == 2


def test_special_values_stay_in_their_row_and_channel():
    """NaN and infinities past a row's end change nothing; inside, they stay in their row and channel."""
    c = (3, 40, 70, 16, 1, "bf16", 1, None, False, True, True, True)
    v, dY, dYh, _ = _scan_case(c, seed=7)
    ln = torch.tensor([40, 13, 0], dtype=torch.int32)
    clean = _scan_run(c, v, dY, dYh, ln)
    dirty = {k: None if t is None else t.clone() for k, t in v.items()}
    dyd = dY.clone()
    for k in ("X", "dt", "B", "C", "Z"):
        dirty[k][1, 13:] = float("nan")
        dirty[k][2] = float("inf")
    dyd[1, 13:] = float("nan")
    got = _scan_run(c, dirty, dyd, dYh, ln)
    for k in clean:
        assert torch.equal(got[k], clean[k]), k
    for k in ("Y", "dX", "ddt", "dZ", "dB", "dC"):
        assert not got[k][1, 13:].any() and not got[k][2].any(), k
    dirty = {k: None if t is None else t.clone() for k, t in v.items()}
    dirty["X"][0, 20, 5] = float("nan")
    got = _scan_run(c, dirty, dY, dYh, ln)
    Y, want = got["Y"].clone(), clean["Y"]
    assert Y[0, 20:, 5].isnan().all()
    Y[0, 20:, 5] = want[0, 20:, 5]
    assert torch.equal(Y, want)
    x = v["X"].clone()
    x[0, 3, 4] = float("nan")
    plan = orc.rnn_ssm_create(70, layout=1)
    orc.rnn_ssm_set_io_type(plan, "bf16")
    W = torch.randn(70, 4, generator=torch.Generator().manual_seed(0)).cuda()
    a, _ = orc.ssm_conv(plan, v["X"].cuda(), W)
    b, _ = orc.ssm_conv(plan, x.cuda(), W)
    assert b[0, 3:7, 4].isnan().all()
    b[0, 3:7, 4] = a[0, 3:7, 4]
    assert torch.equal(a, b)


def test_extreme_steps():
    """Steps so large that the state is forgotten, so small that nothing enters, and a softplus past its knee."""
    N, S, D, M = 1, 5, 4, 16
    r = _gen(3)
    v = dict(X=r(N, S, D), dt=torch.zeros(N, S, D), A=-torch.exp(r(D, M)), B=r(N, S, 1, M), C=r(N, S, 1, M), D=r(D),
             Z=None, dt_bias=torch.tensor([60.0, -60.0, 25.0, -20.0]), h0=r(N, D, M))
    c = (N, S, D, M, 1, "f32", 1, None, True, False, True, True)
    dY, dYh = r(N, S, D), r(N, D, M)
    _check_scan(c, v, dY, dYh, None, _scan_run(c, v, dY, dYh, None))


def test_no_steps_and_no_rows():
    D, M, K = 12, 16, 4
    plan = orc.rnn_ssm_create(D, state_size=M, conv_width=K, layout=1)
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    for N, S in ((3, 0), (0, 5), (0, 0)):
        h0, st = torch.randn(N, D, M, device="cuda"), torch.randn(N, K - 1, D, device="cuda")
        A, W = -torch.ones(D, M, device="cuda"), torch.randn(D, K, device="cuda")
        args = (z(N, S, D), z(N, S, D), A, z(N, S, 1, M), z(N, S, 1, M), z(D), z(N, S, D), z(D), None, h0)
        Y, Yh, saved = orc.ssm_scan(plan, *args, save=True)
        assert Y.shape == (N, S, D) and torch.equal(Yh, h0)
        dYh = torch.randn_like(h0)
        g = orc.ssm_scan_grad(plan, z(N, S, D), saved, *args, dY_h=dYh)
        assert torch.equal(g["d_initial_h"], dYh)
        assert not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))
        Y, state = orc.ssm_conv(plan, z(N, S, D), W, z(D), None, st)
        assert torch.equal(state, st)
        g = orc.ssm_conv_grad(plan, z(N, S, D), z(N, S, D), W, z(D), None, st, st)
        assert torch.equal(g["d_initial_state"], st) and not g["dW"].any() and not g["dbias"].any()
    orc.rnn_ssm_conv_step(plan, z(0, D), z(D, K), z(D), z(0, K - 1, D), z(0, D))
    orc.rnn_ssm_scan_step(plan, z(0, D), z(0, D), z(D, M), z(0, 1, M), z(0, 1, M), z(0, D, M), z(0, D))
    orc.rnn_ssm_sync(plan)


@pytest.mark.parametrize("bad", [-1, 41])
def test_bad_lengths_are_reported(bad):
    c = (3, 40, 16, 16, 1, "f32", 1, None, False, True, True, True)
    v, dY, dYh, _ = _scan_case(c)
    ln = torch.tensor([40, bad, 7], dtype=torch.int32)
    with pytest.raises(orc.RNNError) as e:
        _scan_run(c, v, dY, dYh, ln)
    assert e.value.status == 2
    plan = orc.rnn_ssm_create(16, layout=1)
    Y, _ = orc.ssm_conv(plan, v["X"].cuda(), torch.ones(16, 4, device="cuda"), None, ln.cuda())
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_sync(plan)
    good, _ = orc.ssm_conv(plan, v["X"].cuda(), torch.ones(16, 4, device="cuda"), None,
                           torch.tensor([40, 0 if bad < 0 else 40, 7], dtype=torch.int32).cuda())
    orc.rnn_ssm_sync(plan)
    assert torch.equal(Y, good)


def test_other_streams_share_a_plan():
    """Calls of one plan on two streams in turn: the scratch of the first is not overwritten by the second."""
    c = (2, 80, 264, 16, 1, "f32", 1, None, False, True, True, True)
    v, dY, dYh, _ = _scan_case(c)
    want = _scan_run(c, v, dY, dYh, None)
    plan = orc.rnn_ssm_create(264, layout=1)
    cu = {k: None if t is None else t.cuda() for k, t in v.items()}
    args = (cu["X"], cu["dt"], cu["A"], cu["B"], cu["C"], cu["D"], cu["Z"], cu["dt_bias"])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dYc, dYhc = dY.cuda(), dYh.cuda()
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            Y, Yh, saved = orc.ssm_scan(plan, *args, save=True)
            outs.append((Y, saved, orc.ssm_scan_grad(plan, dYc, saved, *args, dY_h=dYhc)))
    torch.cuda.synchronize()
    for Y, _, g in outs:
        assert torch.equal(Y, want["Y"])
        for k in g:
            assert torch.equal(g[k], want[k]), k


def test_capture_and_replay():
    """A token's calls captured once and replayed: each replay advances the states."""
    N, D, M, K = 2, 64, 16, 4
    r = _gen(1)
    plan = orc.rnn_ssm_create(D, state_size=M, conv_width=K)
    x, W, b = r(N, D).cuda(), r(D, K).cuda(), r(D).cuda()
    A, B, C, dt, Z = -torch.exp(r(D, M)).cuda(), r(N, 1, M).cuda(), r(N, 1, M).cuda(), r(N, D).cuda(), r(N, D).cuda()
    def step(state, H, u, y):  # noqa: E306
        orc.rnn_ssm_conv_step(plan, x, W, b, state, u)
        orc.rnn_ssm_scan_step(plan, u, dt, A, B, C, H, y, None, Z)
    state, H, u, y = r(N, K - 1, D).cuda(), r(N, D, M).cuda(), torch.empty(N, D, device="cuda"), torch.empty(N, D, device="cuda")
    s2, h2, u2, y2 = state.clone(), H.clone(), u.clone(), y.clone()
    step(state.clone(), H.clone(), u, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(state, H, u, y)
    for _ in range(3):
        g.replay()
        step(s2, h2, u2, y2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(H, h2) and torch.equal(state, s2)


def test_binding_refuses():
    D = 8
    plan = orc.rnn_ssm_create(D, layout=1)
    x, W = torch.zeros(2, 3, D, device="cuda"), torch.zeros(D, 4, device="cuda")
    for X, w, err in ((x.half(), W, TypeError), (x.cpu(), W, (TypeError, ValueError)), (x, W[:, :3].contiguous(), ValueError),
                      (x[..., :4], W, ValueError), (x, W.double(), TypeError), (x.transpose(1, 2), W, ValueError),
                      (torch.zeros(1, device="cuda").expand(2, 3, D), W, ValueError), (x[0], W, ValueError)):
        with pytest.raises(err):
            orc.rnn_ssm_conv(plan, X, w, Y=torch.empty_like(x))
    bc = torch.zeros(2, 3, 1, 16, device="cuda")
    with pytest.raises(orc.RNNError):
        orc.rnn_ssm_scan(plan, x, x, torch.zeros(D, 16, device="cuda"), bc, bc)      # no Y
    with pytest.raises(ValueError):
        orc.rnn_ssm_scan(plan, x, x, torch.zeros(D, 16, device="cuda"), bc[..., :8], bc, Y=torch.empty_like(x))
    with pytest.raises(ValueError):
        orc.ssm_scan(plan, x, x[:, :2], torch.zeros(D, 16, device="cuda"), bc, bc)
