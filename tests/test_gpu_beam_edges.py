"""Beam search where everyday calls do not lead: masks of a type's lowest value, many equal logits, rows shared by an item's
beams and cut in parts."""
import math

import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


@pytest.mark.parametrize("V", [50, 5000, 50001])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_a_row_of_a_masks_lowest_value_is_uniform(io, V):
    """Each of its tokens has -log V, which beams of lower scores with a likely token beat.  The sum is one of ones, exact in 32
    bits, and the likely tokens' rows sum to 1 within V e^-80 (or are exact): scores are rounded once, by 2^-24 of themselves."""
    B = 3
    plan = orc.rnn_beam_create(B)
    x = torch.zeros(2 * B, V, dtype=DT[io])
    x[0] = torch.finfo(DT[io]).min
    x[1, 7] = x[2, 9] = 80.0
    x[B:] = torch.finfo(DT[io]).min
    scores = torch.tensor([[0.0, -1.0, -2.0], [-3.0, -1.0, -2.0]])
    step = orc.beam_select(plan, x.cuda(), scores.cuda())
    assert step.parents.tolist() == [[1, 2, 0], [1, 1, 1]] and step.ids.tolist() == [[7, 9, 0], [0, 1, 2]]
    u = math.log(V)
    want = torch.tensor([[-1.0, -2.0, -u], [-1.0 - u] * 3], dtype=torch.float64)
    assert ((step.scores.cpu().double() - want).abs() <= 2.0 ** -24 * want.abs() + 1e-12).all()


def test_beams_whose_score_is_not_finite_have_no_candidates():
    B, V = 4, 30
    plan = orc.rnn_beam_create(B, end_id=3)
    x = torch.randn(B, V)
    scores = torch.tensor([[float("inf"), -1.0, float("nan"), float("inf")]])
    done = torch.tensor([[False, False, True, True]])
    step = orc.beam_select(plan, x.cuda(), scores.cuda(), done.cuda())
    assert step.parents.tolist() == [[1] * 4]
    assert step.ids[0].tolist() == x[1].topk(4).indices.tolist()
    x[1] = NEG              # all are -inf: the lowest beam's lowest tokens
    step = orc.beam_select(plan, x.cuda(), scores.cuda(), done.cuda())
    assert step.parents.tolist() == [[0] * 4] and step.ids.tolist() == [[0, 1, 2, 3]] and (step.scores == NEG).all()


def _check(plan, logits, scores, shared=False):
    """Against all candidates in 64 bits: parents and tokens equal, scores within those of sums of at most 200 roundings a part."""
    items, B = scores.shape
    step = orc.beam_select(plan, logits.cuda(), scores.cuda())
    x = logits.double()
    x = x[:, None].expand(items, B, -1) if shared else x.view(items, B, -1)
    parents, ids, new, _ = ref.beam(x, scores, None, plan.end_id)
    assert torch.equal(step.parents.cpu().long(), parents) and torch.equal(step.ids.cpu().long(), ids)
    got = step.scores.cpu().double()
    assert ((got == new) | ((got - new).abs() <= 2.0 ** -24 * new.abs() + 200 * 2.0 ** -24)).all()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,V", [(1, 3000), (4, 3000), (32, 3000), (5, 40001)])
def test_more_equal_logits_than_the_list_holds(B, V, io):
    """An untrained model's row, rows of few different logits, rows of one large one among equals, and rows that begin off
    a boundary: more logits reach the bound than the list of a part holds."""
    g = torch.Generator().manual_seed(V + B)
    plan = orc.rnn_beam_create(B)
    x = torch.zeros(2 * B, V, dtype=DT[io])
    scores = torch.arange(2.0 * B).view(2, B) * -0.01
    _check(plan, x, scores)
    x = torch.randint(0, 3, (2 * B, V), generator=g).to(DT[io])
    _check(plan, x, scores)
    x[:] = -1.0
    x[:, V // 2], x[:, V - 1] = 0.0, 0.5
    _check(plan, x, scores)
    wide = torch.zeros(2 * B, V + 5, dtype=DT[io], device="cuda")
    wide[:, 3:3 + V] = x.cuda()
    step, same = orc.beam_select(plan, wide[:, 3:3 + V], scores.cuda()), orc.beam_select(plan, x.cuda(), scores.cuda())
    assert torch.equal(step.ids, same.ids) and torch.equal(step.parents, same.parents)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_parts_with_fewer_tokens_than_beams(io):
    """A mask that leaves a few tokens, all in some of a row's parts."""
    B, V = 8, 30000
    plan = orc.rnn_beam_create(B)
    x = torch.full((B, V), NEG, dtype=DT[io])
    scores = torch.arange(float(B))[None] * -0.37
    for b in range(B):
        x[b, 9000 + b:9000 + 2 * b + 1] = torch.arange(float(b + 1))
    x[3, 29999] = 2.0
    _check(plan, x, scores)
    x[1:] = NEG             # one beam, one token, and then the lowest places
    _check(plan, x, scores)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [5000, 50001])
def test_a_row_shared_by_beams_and_cut_in_parts(V, io):
    g = torch.Generator().manual_seed(V)
    B, items = 6, 2
    plan = orc.rnn_beam_create(B)
    x = (3 * torch.randn(items, V, generator=g)).to(DT[io])
    scores = -torch.rand(items, B, generator=g)
    _check(plan, x, scores, shared=True)
    scores[:, 1:] = NEG     # a first step
    _check(plan, x, scores, shared=True)
    wide = orc.beam_select(plan, x.repeat_interleave(B, 0).cuda(), scores.cuda())
    one = orc.beam_select(plan, x.cuda(), scores.cuda())
    assert torch.equal(one.ids, wide.ids) and torch.equal(one.parents, wide.parents)


def test_a_tensor_without_rows_is_refused():
    plan = orc.rnn_beam_create(2)
    parents, slots = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(slots=slots)):
        with pytest.raises(ValueError):
            orc.rnn_beam_reorder(plan, parents, [torch.zeros((), device="cuda")], **kw)
