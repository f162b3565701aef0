"""The gated delta rule, layer normalisation and beam search where their documents allow more than everyday calls: plans
shared by streams, captured long rows, more heads and items than a grid's dimension holds, operands of any magnitude."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu


def _inputs(N, S, H, HK, DK, DV, seed=0, decay=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda t: 0.99 * t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    return [unit(r(N, S, HK, DK)), unit(r(N, S, HK, DK)), r(N, S, H, DV), -decay * torch.rand(N, S, H, generator=g),
            torch.rand(N, S, H, generator=g)], r(N, H, DK, DV), r(N, S, H, DV), r(N, H, DK, DV)


def test_streams_that_share_a_plan():
    """Calls of one plan on two streams in turn: the scratch, which both use, is handed over in order."""
    plan = orc.rnn_delta_create(3, 24, 40, 1, layout=1)
    norm = orc.rnn_norm_create(40)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    cases, want = [], []
    for k, (N, S) in enumerate(((2, 500), (3, 300))):
        ins, state, dY, _ = _inputs(N, S, 3, 1, 24, 40, seed=k)
        cases.append(([t.cuda() for t in ins], state.cuda(), dY.cuda()))
    w = torch.linspace(0.5, 1.5, 40, device="cuda")

    def both(ins, state, dY, stream):
        Y, end, saved = orc.delta_rule(plan, *ins, None, state, save=True, stream=stream)
        out = orc.delta_rule_grad(plan, dY, saved, *ins, None, state, stream=stream)
        Z, stats = orc.layer_norm(norm, Y, w, stream=stream)
        return [Y, end, *out.values(), Z, *orc.layer_norm_grad(norm, dY, Y, stats, w, w, stream=stream).values()]
    for c in cases:
        want.append(both(*c, None))
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for c, side in zip(cases, sides):
            got.append(both(*c, side))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2])), k


def test_a_captured_long_row():
    """A row long enough to be cut, replayed with other inputs in the same places."""
    ins, state, _, _ = _inputs(1, 4500, 2, 1, 32, 48)
    other, state2, _, _ = _inputs(1, 4500, 2, 1, 32, 48, seed=1)
    plan, plain = (orc.rnn_delta_create(2, 32, 48, 1, layout=1) for _ in range(2))
    held, st = [t.cuda() for t in ins], state.cuda()
    Y, end = torch.empty_like(held[2]), torch.empty_like(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        orc.rnn_delta_rule(plan, *held, None, st, Y, end)
    assert orc.rnn_delta_last_launch_count(plan) > 2        # (cut)
    for a, s in ((ins, state), (other, state2)):
        for t, x in zip(held, a):
            t.copy_(x)
        st.copy_(s)
        graph.replay()
        want = orc.delta_rule(plain, *held, None, st)
        assert torch.equal(Y, want[0]) and torch.equal(end, want[1])


def test_more_heads_than_a_grids_dimension():
    N, S, H, DK, DV = 33001, 2, 2, 4, 5
    ins, state, dY, d_state = _inputs(N, S, H, H, DK, DV)
    plan = orc.rnn_delta_create(H, DK, DV, layout=1)
    gpu = [t.cuda() for t in ins]
    Y, end, saved = orc.delta_rule(plan, *gpu, None, state.cuda(), save=True)
    want = ref.delta(*[t.double() for t in ins], None, state.double(), plan.scale)
    ref.close(Y, want[0], S, DK + 128, "f32", "Y")
    ref.close(end, want[1], S, DK + 128, "f32", "state")
    out = orc.delta_rule_grad(plan, dY.cuda(), saved, *gpu, None, state.cuda(), d_state=d_state.cuda())
    grads = ref.delta_grad(dY.double(), d_state.double(), *[t.double() for t in ins], None, state.double(), plan.scale)
    for name, t in out.items():
        ref.close(t, grads[name], 3 * S, DK + 128 + DV, "f32", name)
    one = [t[:, 0].contiguous() for t in gpu]
    st, y = state.cuda(), torch.empty(N, H, DV, device="cuda")
    orc.rnn_delta_step(plan, *one, st, y)
    want = ref.delta(*[t[:, :1].double() for t in ins], None, state.double(), plan.scale)
    ref.close(y[:, None], want[0], 1, DK + 128, "f32", "token")
    ref.close(st, want[1], 1, DK + 128, "f32", "token's state")
    orc.rnn_delta_sync(plan)


@pytest.mark.parametrize("S", [70, 4500])
def test_powers_of_two_change_no_bits(S):
    """Operands are scaled to their largest values: results of inputs times powers of two are those times powers of two."""
    ins, state, dY, d_state = _inputs(1, S, 2, 1, 40, 33, seed=2)
    plan = orc.rnn_delta_create(2, 40, 33, 1, layout=1)

    def run(q, v, dy, ds):
        a = [ins[0] * q, ins[1], ins[2] * v, ins[3], ins[4]]
        a, s = [t.cuda() for t in a], (state * v).cuda()
        Y, end, saved = orc.delta_rule(plan, *a, None, s, save=True)
        return dict(Y=Y, end=end, **orc.delta_rule_grad(plan, (dY * dy).cuda(), saved, *a, None, s, d_state=(d_state * ds).cuda()))
    plain, moved = run(1, 1, 1, 1), run(2.0 ** -30, 2.0 ** 40, 2.0 ** -40, 2.0 ** -70)
    by = dict(Y=10, end=40, dQ=0, dK=-30, dV=-70, dg=-30, dbeta=-30, d_initial_state=-70)
    for name, t in plain.items():
        assert torch.equal(t * 2.0 ** by[name], moved[name]), name


def test_more_items_than_a_grids_dimension():
    g = torch.Generator().manual_seed(4)
    items, B, V = 70001, 2, 5
    plan = orc.rnn_beam_create(B)
    logits, scores = torch.randn(items * B, V, generator=g).cuda(), torch.randn(items, B, generator=g).cuda()
    step = orc.beam_select(plan, logits, scores)
    every = (torch.log_softmax(logits.double(), 1).view(items, B, V) + scores.double()[:, :, None]).view(items, -1)
    best = every.topk(B, 1)
    # (of 700010 candidates some may lie closer together than lse's error)
    far = (every.topk(B + 1, 1).values.diff(dim=1).abs() > 1e-5).all(1)
    assert int(far.sum()) > 0.99 * items
    assert torch.equal((step.parents.long() * V + step.ids)[far], best.indices[far])
    t = torch.randn(items * B, 6, generator=g).cuda()
    rows = (step.parents.long() + torch.arange(items, device="cuda")[:, None] * B).view(-1)
    want = t[rows]
    orc.rnn_beam_reorder(plan, step.parents, [t])
    assert torch.equal(t, want)
    orc.rnn_beam_sync(plan)


@pytest.mark.parametrize("B", [4, 12])
def test_rows_that_stay_among_rows_that_move(B):
    """In place, into other memory, and at slots: a row that becomes itself is there all the same."""
    plan = orc.rnn_beam_create(B)
    g = torch.Generator().manual_seed(B)
    parents = torch.arange(B, dtype=torch.int32).repeat(3, 1)
    parents[1, B // 2:] = 0
    parents[2] = torch.randint(0, B, (B,), generator=g)
    t = torch.randn(3 * B, 37, generator=g)
    rows = (parents.long() + torch.arange(3)[:, None] * B).view(-1)
    x, p = t.cuda(), parents.cuda()
    y, = orc.beam_reorder(plan, p, [x])
    assert torch.equal(y.cpu(), t[rows])
    slots = torch.randperm(5 * B, generator=g)[:3 * B]
    pool = torch.randn(5 * B, 37, generator=g)
    want = pool.clone()
    want[slots] = pool[slots][rows]
    pool = pool.cuda()
    orc.rnn_beam_reorder(plan, p, [pool], slots=slots.int().cuda())
    assert torch.equal(pool.cpu(), want)
    orc.rnn_beam_reorder(plan, p, [x])
    assert torch.equal(x.cpu(), t[rows])
    orc.rnn_beam_sync(plan)
