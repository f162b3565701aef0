"""The 64-bit reference of a step of beam search where its logits are far from zero."""
import math

import torch

import delta_ref64 as ref


def test_a_row_of_a_masks_lowest_value_is_uniform():
    V = 50
    x = torch.full((1, 2, V), float(torch.finfo(torch.float32).min), dtype=torch.float64)
    x[0, 1] = 0.0
    x[0, 1, 4] = 80.0
    parents, ids, new, _ = ref.beam(x, torch.tensor([[0.0, -1.0]]), None, -1)
    assert parents.tolist() == [[1, 0]] and ids.tolist() == [[4, 0]]
    assert torch.allclose(new[0], torch.tensor([-1.0, -math.log(V)], dtype=torch.float64), rtol=1e-14)
