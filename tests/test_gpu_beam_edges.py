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
