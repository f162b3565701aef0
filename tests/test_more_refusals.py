"""Refusals of the gated delta rule, layer normalisation and beam search that need no GPU.  Arguments stand in the
order of the header's structures; the addresses must not be read."""
import ctypes
import struct

import pytest

import onnx_recurrent_gb300 as orc

AT, FAR = 4096, 1 << 30


@pytest.fixture(scope="module")
def lib():
    orc.build()
    from onnx_recurrent_gb300 import beam, delta, norm
    delta._load(), norm._load()
    return beam._load()


def _run(fn, plan, fields):
    return fn(plan.handle, struct.pack(f"{len(fields)}q", *fields))


def _refused(fn, plan, fields, text):
    assert _run(fn, plan, fields) == 1, text
    assert text in orc.rnn_last_error(), orc.rnn_last_error()


def test_plans(lib):
    for a in [dict(heads=0), dict(heads=4, key_heads=3), dict(heads=4, key_heads=0), dict(heads=1, key_size=0), dict(heads=1, key_size=129),
              dict(heads=1, value_size=0), dict(heads=1, value_size=1025), dict(heads=1, layout=2), dict(heads=1, scale=float("nan")),
              dict(heads=2 ** 30, value_size=4)]:
        with pytest.raises(orc.RNNError):
            orc.rnn_delta_create(**a)
    for a in [(0,), (32769,), (8, -1.0), (8, float("nan")), (8, float("inf"))]:
        with pytest.raises(orc.RNNError):
            orc.rnn_norm_create(*a)
    for a in [(0,), (33,), (4, -2), (4, 2 ** 31)]:
        with pytest.raises(orc.RNNError):
            orc.rnn_beam_create(*a)


D3 = (AT, 0, 0)


def delta_run(lens=0, init=0, Y=(FAR, 0, 0), final=0, saved=0, S=5, N=2, ins=(D3,) * 5):
    return [S, N, *[x for v in ins for x in v], lens, init, *Y, final, saved, 0]


def test_delta_arguments(lib):
    p = orc.rnn_delta_create(2, 4, 8)
    f = lib.rnn_delta_rule
    for i, name in enumerate(("Q", "K", "V", "g", "beta")):
        ins = [D3] * 5
        ins[i] = (0, 0, 0)
        _refused(f, p, delta_run(ins=ins), f"{name} is NULL")
        ins[i] = (AT + 1, 0, 0)
        _refused(f, p, delta_run(ins=ins), f"{name} is not aligned")
        ins[i] = (AT, -1, 64)
        _refused(f, p, delta_run(ins=ins), f"{name} has a negative stride")
    _refused(f, p, delta_run(Y=(0, 0, 0)), "Y is NULL")
    _refused(f, p, delta_run(S=-1), "seq_length")
    for ss, bs in [(0, 64), (64, 0), (8, 64), (16, 40), (20, 16), (16, 79)]:
        _refused(f, p, delta_run(Y=(FAR, ss, bs)), "share memory")
    _refused(f, p, delta_run(init=AT, final=AT + 64), "overlap in part")
    _refused(f, p, delta_run(saved=AT + 2), "saved is not aligned")
    assert _run(f, p, delta_run(N=0)) == 0 and _run(f, p, delta_run(S=0)) == 0
    g = lib.rnn_delta_rule_grad
    base = lambda outs, saved=AT, dend=0, dinit=0: [5, 2, *D3, *D3 * 5, 0, saved, dend, *[x for o in outs for x in o], dinit, 0]  # noqa: E731
    none = [(0, 0, 0)] * 5
    _refused(g, p, base(none, saved=0), "saved is NULL")
    _refused(g, p, base(none, dend=AT, dinit=AT + 64), "overlap in part")
    for i, name in enumerate(("dQ", "dK", "dV", "dg", "dbeta")):
        outs = list(none)
        outs[i] = (FAR, 1, 1)
        _refused(g, p, base(outs), "share memory")
    st = lib.rnn_delta_step
    step = lambda state=AT, out=AT, slots=0, n=3, Y=D3: [2, n, *D3 * 5, state, out, slots, *Y, 0]  # noqa: E731
    _refused(st, p, step(state=0), "state is NULL")
    _refused(st, p, step(out=0), "state_out is NULL")
    _refused(st, p, step(out=AT + 128), "overlap in part")
    _refused(st, p, step(slots=AT, n=0), "n_slots")
    _refused(st, p, step(Y=(FAR, 0, 8)), "share memory")


def test_norm_arguments(lib):
    p = orc.rnn_norm_create(16)
    f, g = lib.rnn_layer_norm, lib.rnn_layer_norm_grad
    _refused(f, p, [3, 0, 0, 0, 0, FAR, 0, 0, 0], "X is NULL")
    _refused(f, p, [3, AT, 0, 0, 0, 0, 0, 0, 0], "Y is NULL")
    _refused(f, p, [3, AT, -16, 0, 0, FAR, 0, 0, 0], "negative stride")
    _refused(f, p, [3, AT, 0, 0, 0, FAR, 15, 0, 0], "share memory")
    _refused(f, p, [3, AT, 0, 0, 0, AT + 64, 0, 0, 0], "overlap in part")
    _refused(f, p, [3, AT, 16, 0, 0, AT, 32, 0, 0], "overlap in part")
    _refused(f, p, [3, AT, 31, 0, 0, AT + 64, 31, 0, 0], "overlap in part")
    _refused(f, p, [3, AT, 0, AT + 1, 0, FAR, 0, 0, 0], "W is not aligned")
    _refused(f, p, [-1, AT, 0, 0, 0, FAR, 0, 0, 0], "rows")
    assert _run(f, p, [0] * 9) == 0
    _refused(g, p, [3, AT, 0, AT, 0, 0, 0, FAR, 0, 0, 0, 0], "stats is NULL")
    _refused(g, p, [3, AT, 0, 2 * FAR, 0, AT, 0, AT + 4, 0, 0, 0, 0], "dY and dX overlap")
    _refused(g, p, [3, 2 * FAR, 0, AT, 0, AT, 0, AT + 4, 0, 0, 0, 0], "X and dX overlap")


def test_beam_arguments(lib):
    p, open_ = orc.rnn_beam_create(4, end_id=9), orc.rnn_beam_create(4)
    f = lib.rnn_beam_select
    ok = [2, 10, 0, AT, 0, 0, AT, 0, FAR, FAR + 64, FAR + 128, 0, 0]

    def but(**kw):
        names = "items vocab io logits stride shared scores finished parents ids new fin stream".split()
        return [kw.get(n, v) for n, v in zip(names, ok)]
    _refused(f, p, but(vocab=0), "vocab")
    _refused(f, p, but(vocab=9), "end_id")
    _refused(f, p, but(io=3), "io type")
    _refused(f, p, but(stride=9), "row_stride")
    _refused(f, p, but(shared=2), "shared")
    _refused(f, open_, but(finished=AT), "without an end_id")
    for n in ("logits", "scores", "parents", "ids"):
        _refused(f, p, but(**{n: 0}), "NULL")
    _refused(f, p, but(new=0), "new_scores is NULL")
    _refused(f, p, but(new=AT + 4), "scores and new_scores overlap")
    _refused(f, p, but(finished=AT, fin=AT + 1), "finished and new_finished overlap")
    assert _run(f, p, but(items=0)) == 0
    r = lib.rnn_beam_reorder
    table = lambda *rows: ctypes.create_string_buffer(struct.pack(f"{3 * len(rows)}q", *[x for t in rows for x in t]))  # noqa: E731
    one = table((AT, AT + 8, 16))
    _refused(r, p, [2, 1, 0, AT, 0, ctypes.addressof(one), 0], "overlap in part")
    one = table((AT, 0, 16))
    _refused(r, p, [2, 1, 0, AT, 0, ctypes.addressof(one), 0], "out is NULL")
    one = table((AT, FAR, -16))
    _refused(r, p, [2, 1, 0, AT, 0, ctypes.addressof(one), 0], "row_bytes")
    _refused(r, p, [2, 1, 0, 0, 0, AT, 0], "parents is NULL")
    _refused(r, p, [2, 1, 0, AT, 0, 0, 0], "tensors is NULL")
    _refused(r, p, [2, 1, 0, AT, AT, AT, 0], "n_slots")
    assert _run(r, p, [2, 0, 0, 0, 0, 0, 0]) == 0


def test_the_binding_checks_shapes_and_types():
    import torch
    p = orc.rnn_delta_create(2, 4, 8, layout=1)
    t = torch.zeros(1, 3, 2, 4)
    with pytest.raises(TypeError):
        orc.delta_rule(p, t, t, torch.zeros(1, 3, 2, 8), torch.zeros(1, 3, 2), torch.zeros(1, 3, 2))
    with pytest.raises(TypeError):
        orc.layer_norm(orc.rnn_norm_create(4), torch.zeros(3, 4))
    with pytest.raises(TypeError):
        orc.beam_select(orc.rnn_beam_create(2), torch.zeros(2, 4), torch.zeros(1, 2))


def test_sizes_past_counting(lib):
    """Sizes whose images would not be counted in 64 bits, each of which is in range by itself."""
    p = orc.rnn_delta_create(1024, 128, 1024)
    assert orc.rnn_delta_saved_size(p, 2 ** 30, 2 ** 20) == -1
    assert orc.rnn_delta_saved_size(p, 2 ** 20, 2 ** 10) > 0
    a = delta_run()
    a[0], a[1] = 2 ** 30, 2 ** 20
    assert _run(lib.rnn_delta_rule, p, a) != 0 and "2^31 or more" in orc.rnn_last_error()


def test_tensors_reordered_at_once_lie_apart(lib):
    """Blocks of all tensors run side by side: a tensor given twice would be reordered while it is read."""
    p = orc.rnn_beam_create(4)
    r = lib.rnn_beam_reorder
    table = lambda *rows: ctypes.create_string_buffer(struct.pack(f"{3 * len(rows)}q", *[x for t in rows for x in t]))  # noqa: E731
    # 8 rows of 16 bytes each: 128 bytes a tensor; parents 32 bytes at AT
    for second in [(FAR, FAR, 16), (FAR, 2 * FAR, 16), (2 * FAR, FAR, 16), (FAR + 64, FAR + 64, 16), (2 * FAR, FAR + 127, 16)]:
        both = table((FAR, FAR, 16), second)
        _refused(r, p, [2, 2, 0, AT, 0, ctypes.addressof(both), 0], "tensors 0 and 1 overlap")
    one = table((FAR, AT + 16, 16))
    _refused(r, p, [2, 1, 0, AT, 0, ctypes.addressof(one), 0], "overlaps parents")
    one = table((FAR, 2 * FAR, 16))
    _refused(r, p, [2, 1, 100, AT, 2 * FAR + 1596, ctypes.addressof(one), 0], "overlaps parents or slots")
