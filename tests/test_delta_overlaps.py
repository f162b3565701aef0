"""Outputs of the gated delta rule that lie on inputs or on one another are refused, in place of results that depend on the
order of blocks; parts of wider rows side by side are not.  Addresses of refused calls must not be read."""
import struct

import pytest
import torch

import onnx_recurrent_gb300 as orc

FAR = 1 << 32
S, N, H, HK, DK, DV = 5, 2, 2, 1, 4, 8      # layout 0, fp32


@pytest.fixture(scope="module")
def lib():
    orc.build()
    from onnx_recurrent_gb300 import delta
    return delta._load()


def _refused(fn, plan, fields, text):
    assert fn(plan.handle, struct.pack(f"{len(fields)}q", *fields)) == 1, text
    assert text in orc.rnn_last_error(), (text, orc.rnn_last_error())


INS = {n: (FAR * (i + 1), 0, 0) for i, n in enumerate(("Q", "K", "V", "g", "beta"))}


def run(lens=FAR * 6, init=FAR * 7, Y=(FAR * 8, 0, 0), final=FAR * 9, saved=FAR * 10, **ins):
    return [S, N, *[x for v in {**INS, **ins}.values() for x in v], lens, init, *Y, final, saved, 0]


def grad(lens=FAR * 6, saved=FAR * 7, dend=FAR * 8, dinit=FAR * 9, dY=(FAR * 10, 0, 0), ins={}, **outs):
    at = {n: (FAR * (11 + i), 0, 0) for i, n in enumerate(("dQ", "dK", "dV", "dg", "dbeta"))}
    return [S, N, *dY, *[x for v in {**INS, **ins}.values() for x in v], lens, saved, dend, *[x for v in {**at, **outs}.values() for x in v], dinit, 0]


def test_runs(lib):
    p, f = orc.rnn_delta_create(H, DK, DV, HK), lib.rnn_delta_rule
    rows = S * N * H * DV * 4
    _refused(f, p, run(Y=INS["V"]), "Y overlaps V")
    _refused(f, p, run(Y=(FAR * 3 + rows - 4, 0, 0)), "Y overlaps V")
    _refused(f, p, run(Y=(FAR * 3 - rows + 4, 0, 0)), "Y overlaps V")
    for name in ("Q", "K", "g", "beta"):
        _refused(f, p, run(Y=(INS[name][0] - 64, 0, 0)), f"Y overlaps {name}")
    _refused(f, p, run(Y=(FAR * 6 - 4, 0, 0)), "Y overlaps sequence_lens")
    _refused(f, p, run(Y=(FAR * 7 - 4, 0, 0)), "Y overlaps initial_state")
    _refused(f, p, run(Y=(FAR * 9 - 4, 0, 0)), "Y overlaps final_state")
    _refused(f, p, run(saved=FAR * 8), "saved overlaps Y")
    _refused(f, p, run(saved=FAR * 1 - 16), "saved overlaps Q")
    _refused(f, p, run(final=FAR * 4 - 16), "final_state overlaps g")
    # parts of one wide row: a value into another's part, from either side, and a row further
    wide = 3 * H * DV
    for off in (-H * DV + 1, -1, 0, 1, H * DV - 1, N * wide + 3, -N * wide - 3, wide + H * DV - 1):
        _refused(f, p, run(V=(FAR * 3, N * wide, wide), Y=(FAR * 3 + 4 * off, N * wide, wide)), "Y overlaps V")
    # a dense output amid a wide input's parts
    _refused(f, p, run(V=(FAR * 3, N * wide, wide), Y=(FAR * 3 + 4 * (wide - 3), 0, 0)), "Y overlaps V")


def test_gradients(lib):
    p, f = orc.rnn_delta_create(H, DK, DV, HK), lib.rnn_delta_rule_grad
    _refused(f, p, grad(dV=INS["V"]), "dV overlaps V")
    _refused(f, p, grad(dV=(FAR * 10, 0, 0)), "dV overlaps dY")
    _refused(f, p, grad(dQ=INS["Q"]), "dQ overlaps Q")
    _refused(f, p, grad(dK=(FAR * 11, 0, 0)), "dK overlaps dQ")
    _refused(f, p, grad(dg=INS["g"]), "dg overlaps g")
    _refused(f, p, grad(dbeta=(FAR * 14, 0, 0)), "dbeta overlaps dg")
    _refused(f, p, grad(dbeta=(FAR * 7 + 4, 0, 0)), "dbeta overlaps saved")
    _refused(f, p, grad(dinit=FAR * 3), "d_initial_state overlaps V")
    _refused(f, p, grad(dQ=(FAR * 8, 0, 0)), "dQ overlaps d_final_state")


def test_tokens(lib):
    p, f = orc.rnn_delta_create(H, DK, DV, HK), lib.rnn_delta_step
    step = lambda Y, state=FAR * 6, out=FAR * 6, slots=FAR * 8, n=3: [N, n, *[x for v in INS.values() for x in v], state, out, slots, *Y, 0]  # noqa: E731
    _refused(f, p, step(INS["V"]), "Y overlaps V")
    _refused(f, p, step((FAR * 6 + 4 * (3 * H * DK * DV - 1), 0, 0)), "Y overlaps state")
    _refused(f, p, step((FAR * 8, 0, 0)), "Y overlaps slots")
    _refused(f, p, step((FAR * 9, 0, 0), out=FAR * 5 - 16), "state_out overlaps beta")


@pytest.mark.gpu
def test_parts_of_wide_rows_side_by_side():
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n, s = 3, 70
    for layout in (0, 1):
        p = orc.rnn_delta_create(H, DK, DV, HK, layout=layout)
        lead = (n, s) if layout else (s, n)
        sizes = [HK * DK, HK * DK, H * DV, H * DV]
        wide = 0.3 * r(*lead, sum(sizes) + 5)
        Q, K, V, Y = (t.unflatten(-1, (-1, d)) for t, d in zip(wide[..., 1:1 + sum(sizes)].split(sizes, -1), (DK, DK, DV, DV)))
        small = torch.rand(*lead, 2 * H, generator=g, device="cuda")
        decay, beta = small[..., :H], small[..., H:]
        decay.neg_()
        want, end, saved = orc.delta_rule(p, *(t.contiguous() for t in (Q, K, V, decay, beta)), save=True)
        orc.rnn_delta_rule(p, Q, K, V, decay, beta, Y=Y)
        assert torch.equal(Y, want)
        dY = r(*want.shape)
        grads = orc.delta_rule_grad(p, dY, saved, Q, K, V, decay, beta)
        both, slopes = torch.empty_like(wide), torch.empty_like(small)
        dQ, dK, dV, d4 = (t.unflatten(-1, (-1, d)) for t, d in zip(both[..., 1:1 + sum(sizes)].split(sizes, -1), (DK, DK, DV, DV)))
        d4.copy_(dY)
        orc.rnn_delta_rule_grad(p, d4, saved, Q, K, V, decay, beta, dQ=dQ, dK=dK, dV=dV, dg=slopes[..., :H], dbeta=slopes[..., H:])
        for t, name in ((dQ, "dQ"), (dK, "dK"), (dV, "dV"), (slopes[..., :H], "dg"), (slopes[..., H:], "dbeta")):
            assert torch.equal(t, grads[name]), name
    # tokens: a part of the projection's row takes the output
    p = orc.rnn_delta_create(H, DK, DV, HK)
    wide, small, state = 0.3 * r(n, sum(sizes)), torch.rand(n, 2 * H, generator=g, device="cuda"), r(n, H, DK, DV)
    Q, K, V, Y = (t.unflatten(-1, (-1, d)) for t, d in zip(wide.split(sizes, -1), (DK, DK, DV, DV)))
    out, want = torch.empty_like(state), torch.empty(n, H, DV, device="cuda")
    orc.rnn_delta_step(p, *(t.contiguous() for t in (Q, K, V, -small[:, :H], small[:, H:])), state, want, state_out=out)
    orc.rnn_delta_step(p, Q, K, V, -small[:, :H], small[:, H:], state, Y)
    assert torch.equal(Y, want) and torch.equal(state, out)
