"""Beam search on the GPU against sorting all candidates in 64 bits.  Parents and tokens have to be equal;
scores are rounded once, from sums that err by some 10^-7 (lse's fp32 sum of V terms in a tree)."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


def _check(plan, logits, scores, finished=None, shared=False):
    items, B = scores.shape
    step = orc.beam_select(plan, logits.cuda(), scores.cuda(), None if finished is None else finished.cuda())
    x = logits.double()
    x = x[:, None].expand(items, B, -1) if shared else x.view(items, B, -1)
    parents, ids, new, fin = ref.beam(x, scores, finished, plan.end_id)
    assert torch.equal(step.parents.cpu().long(), parents), "parents"
    assert torch.equal(step.ids.cpu().long(), ids), "ids"
    assert torch.equal(step.finished.cpu(), fin), "finished"
    got = step.scores.cpu().double()
    same = (got == new) | ((got - new).abs() <= 2.0 ** -24 * new.abs() + 1e-6)
    assert same.all(), "scores"
    return step


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1), (2, 4, 3), (3, 2, 100), (5, 8, 1001), (2, 32, 40), (1, 32, 5000), (40, 3, 777), (1, 5, 50001)], ids=str)
def test_selection(size, io):
    items, B, V = size
    g = torch.Generator().manual_seed(V)
    plan = orc.rnn_beam_create(B, end_id=V - 1)
    logits = (2.5 * torch.randn(items * B, V, generator=g)).to(DT[io])
    scores = -10 * torch.rand(items, B, generator=g)
    _check(plan, logits, scores)
    _check(plan, logits, scores, torch.rand(items, B, generator=g) < 0.4)


def test_ties_go_to_the_lowest_beam_then_token():
    plan = orc.rnn_beam_create(4, end_id=2)
    _check(plan, torch.zeros(8, 6), torch.zeros(2, 4))
    x = torch.zeros(4, 300)
    x[1, 200], x[3, 200] = 3.0, 3.0
    _check(plan, x, torch.zeros(1, 4))
    x[:] = torch.tensor([0.0, 1.0]).repeat(150)             # every row the same, many equal logits
    _check(plan, x, torch.tensor([[-1.0, -0.5, -1.0, -0.5]]))


def test_first_step_masks_and_rows_with_nothing():
    g = torch.Generator().manual_seed(1)
    B, V = 4, 50
    plan = orc.rnn_beam_create(B, end_id=0)
    x = torch.randn(3 * B, V, generator=g)
    scores = torch.zeros(3, B)
    scores[0, 1:] = NEG                                     # one beam has begun
    x[B:2 * B] = NEG                                        # an item with nothing left
    x[2 * B:, 3:] = NEG                                     # three tokens a beam
    _check(plan, x, scores)
    x[2 * B] = torch.finfo(torch.float32).min               # a mask of the type's lowest value: a uniform row
    _check(plan, x, scores)
    scores[:] = NEG
    _check(plan, x, scores)


def test_rows_with_nan_and_inf_are_never_taken():
    plan = orc.rnn_beam_create(3, end_id=-1)
    x = torch.randn(6, 20)
    x[0, 4], x[4, 7] = float("nan"), float("inf")
    scores = torch.tensor([[0.0, -50.0, -60.0], [-1.0, 0.0, float("nan")]])
    step = _check(plan, x, scores)
    assert 0 not in step.parents[0].tolist() and step.parents[1].tolist() == [0, 0, 0]


def test_rows_shared_by_beams_or_by_all_and_strides():
    g = torch.Generator().manual_seed(2)
    B, V = 4, 333
    plan = orc.rnn_beam_create(B, end_id=5)
    x, scores = torch.randn(3, V, generator=g), -torch.rand(3, B, generator=g)
    a = _check(plan, x, scores, shared=True)
    wide = x.repeat_interleave(B, 0)
    b = _check(plan, wide, scores)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    big = torch.full((12, V + 9), 50.0)
    big[:, 2:2 + V] = wide
    c = orc.beam_select(plan, big.cuda()[:, 2:2 + V], scores.cuda())
    assert all(torch.equal(p, q) for p, q in zip(c[:2] + c[3:], b[:2] + b[3:]))
    # Rows that start elsewhere in 16 bytes go to other threads, and their exponentials are added in another order.  A thread adds at
    # most 16 pieces of 4 or 8, a warp 5 times, a block 8: 145 roundings of positive terms, so each sum is off by at most 145 *
    # 2^-24, its logarithm by as much, and two of them by 2 * 145 * 2^-24; each score is rounded once more.
    assert ((c.scores - b.scores).abs() <= 290 * 2.0 ** -24 + 2 * 2.0 ** -24 * b.scores.abs()).all()
    one = x[:1].cuda().expand(12, V)
    d = orc.beam_select(plan, one, scores.cuda())
    e = _check(plan, x[:1].expand(12, V).contiguous(), scores)
    assert all(torch.equal(p, q) for p, q in zip(d, e))


def test_scores_and_flags_in_place():
    g = torch.Generator().manual_seed(3)
    plan = orc.rnn_beam_create(4, end_id=1)
    x, scores = torch.randn(8, 90, generator=g).cuda(), -torch.rand(2, 4, generator=g).cuda()
    done = torch.tensor([[True, False, False, True], [False] * 4], device="cuda")
    want = orc.beam_select(plan, x, scores, done)
    p, i = torch.empty_like(want.parents), torch.empty_like(want.ids)
    orc.rnn_beam_select(plan, x, scores, done, p, i, scores, done)
    assert all(torch.equal(a, b) for a, b in zip((p, i, scores, done), want))


@pytest.mark.parametrize("B", [1, 3, 8, 32])
@pytest.mark.parametrize("inner,dtype", [((5, 8), torch.float32), ((7,), torch.float32), ((3,), torch.uint8), ((1000,), torch.bfloat16),
                                         ((2, 3, 1025), torch.float16)], ids=str)
def test_reordering(B, inner, dtype):
    g = torch.Generator().manual_seed(B)
    items = 3
    plan = orc.rnn_beam_create(B)
    a = torch.randint(0, 100, (items * B, *inner), generator=g).to(dtype).cuda()
    b = torch.randint(0, 100, (items * B, 4), generator=g).int().cuda()
    parents = torch.randint(0, B, (items, B), generator=g).int().cuda()
    rows = (parents.long() + torch.arange(items, device="cuda")[:, None] * B).view(-1)
    x, y = orc.beam_reorder(plan, parents, [a, b])
    assert torch.equal(x, a[rows]) and torch.equal(y, b[rows])
    orc.rnn_beam_reorder(plan, parents, [a, b])
    assert torch.equal(a, x) and torch.equal(b, y)
    orc.rnn_beam_sync(plan)


def test_many_tensors_and_slots():
    g = torch.Generator().manual_seed(7)
    B, items = 3, 2
    plan = orc.rnn_beam_create(B)
    parents = torch.tensor([[2, 2, 0], [1, 0, 1]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([9, 4, 0, 7, 2, 5], dtype=torch.int32, device="cuda")
    tensors = [torch.randn(10, 4 + i, generator=g).cuda() for i in range(70)]
    want = []
    for t in tensors:
        w = t.clone()
        w[9], w[4], w[0], w[7], w[2], w[5] = t[0], t[0], t[9], t[2], t[7], t[2]
        want.append(w)
    orc.rnn_beam_reorder(plan, parents, tensors, slots=slots)
    assert orc.rnn_beam_last_launch_count(plan) == 3
    assert all(torch.equal(a, b) for a, b in zip(tensors, want))
    orc.rnn_beam_sync(plan)


def test_bad_parents_and_slots_are_reported_and_left():
    plan = orc.rnn_beam_create(2)
    t = torch.arange(8.0, device="cuda").view(4, 2)
    orc.rnn_beam_reorder(plan, torch.tensor([[1, 2], [-1, 0]], dtype=torch.int32, device="cuda"), [t])
    with pytest.raises(orc.RNNError):
        orc.rnn_beam_sync(plan)
    assert t.tolist() == [[2, 3], [2, 3], [4, 5], [4, 5]]
    t = torch.arange(8.0, device="cuda").view(4, 2)
    slots = torch.tensor([3, 4, -1, 1], dtype=torch.int32, device="cuda")
    orc.rnn_beam_reorder(plan, torch.tensor([[0, 0], [1, 0]], dtype=torch.int32, device="cuda"), [t], slots=slots)
    with pytest.raises(orc.RNNError):
        orc.rnn_beam_sync(plan)
    assert t.tolist() == [[0, 1], [2, 3], [4, 5], [6, 7]]
    orc.rnn_beam_reorder(plan, torch.tensor([[1, 1], [1, 1]], dtype=torch.int32, device="cuda"), [t],
                         slots=torch.tensor([-1, 2, -1, -1], dtype=torch.int32, device="cuda"))
    orc.rnn_beam_sync(plan)


def test_captured_search():
    """Steps replayed from a graph, states behind them, against plain steps."""
    g = torch.Generator().manual_seed(9)
    B, V, items = 4, 500, 3
    logits = torch.randn(items * B, V, generator=g).cuda()

    def steps(plan, scores, done, state, parents, ids):
        orc.rnn_beam_select(plan, logits, scores, done, parents, ids, scores, done)
        orc.rnn_beam_reorder(plan, parents, [state])

    def begin():
        s = torch.zeros(items, B, device="cuda")
        s[:, 1:] = NEG
        return (s, torch.zeros(items, B, dtype=torch.bool, device="cuda"), torch.arange(items * B * 6.0, device="cuda").view(-1, 6),
                torch.empty(items, B, dtype=torch.int32, device="cuda"), torch.empty(items, B, dtype=torch.int32, device="cuda"))
    plain, captured = begin(), begin()
    plan = orc.rnn_beam_create(B, end_id=3)
    for _ in range(3):
        steps(plan, *plain)
    graph, other = torch.cuda.CUDAGraph(), orc.rnn_beam_create(B, end_id=3)
    keep = [t.clone() for t in captured]
    with torch.cuda.graph(graph):
        steps(other, *captured)
    for t, k in zip(captured, keep):
        t.copy_(k)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(plain, captured))
