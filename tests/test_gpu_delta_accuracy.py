"""What the gated delta rule's arithmetic loses, next to the same formulas in plain fp32.

Operands of its products have 22 bits or more, a plain form's 24: each rounding is at most 4 times a plain one's, and the sums take no
more of them, so that errors in norm are within 4 times the plain forms', whose sums and terms are the same (delta_plain32); a group of a few
values is given 8 u of its norm beside.  What is far below the largest of a chunk's operands has a floor, 2^-40 of that: a sum
of terms of such errors stays below 2^-38 of the largest group's norm."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc
from delta_plain32 import chunks, groups, like_plain, plain_errors, steps

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


class Case:
    def __init__(self, N, S, H, HK, DK, DV, io, seed=0, decay=0.05, sizes=None, columns=None, betas=None):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        unit = lambda t: 0.99 * t / t.norm(dim=-1, keepdim=True)  # noqa: E731
        dt = DT[io]
        self.ins = [unit(r(N, S, HK, DK)).to(dt), unit(r(N, S, HK, DK)).to(dt), r(N, S, H, DV), -decay * torch.rand(N, S, H, generator=g),
                    0.1 + 0.9 * torch.rand(N, S, H, generator=g)]
        dY = r(N, S, H, DV)
        self.state, self.d_state = r(N, H, DK, DV), r(N, H, DK, DV)
        if sizes is not None:       # slopes of very different sizes
            dY, self.d_state = dY * sizes[None, :, None, None], 1e-9 * self.d_state
        if columns is not None:     # values of very different sizes
            self.ins[2], self.state = self.ins[2] * columns, self.state * columns
        if betas is not None:       # steps that hardly enter the state
            self.ins[4] = self.ins[4] * betas[None, :, None]
        self.ins[2], self.dY = self.ins[2].to(dt), dY.to(dt)
        self.plan = orc.rnn_delta_create(H, key_size=DK, value_size=DV, key_heads=HK, layout=1)
        orc.rnn_delta_set_io_type(self.plan, io)
        self.io = io

    def run(self):
        a = [t.cuda() for t in self.ins]
        Y, end, saved = orc.delta_rule(self.plan, *a, None, self.state.cuda(), save=True)
        out = orc.delta_rule_grad(self.plan, self.dY.cuda(), saved, *a, None, self.state.cuda(), self.d_state.cuda())
        orc.rnn_delta_sync(self.plan)
        return {n: t.cpu() for n, t in dict(Y=Y, state=end, **out).items()}

    def check(self, size, floor=0.0, forms=(steps, chunks)):
        ins = [*self.ins, self.state, self.dY, self.d_state]
        got, want = self.run(), forms[-1](*(t.double() for t in ins), self.plan.scale)
        plain = plain_errors([*ins, self.plan.scale], want, size, forms=forms)
        for name in want:
            io = self.io if name in ("Y", "dQ", "dK", "dV") else "f32"
            like_plain(name, groups(name, got[name].double(), size), groups(name, want[name], size), plain[name], ref.IO_U[io], floor)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [(2, 200, 4, 2, 128, 128), (3, 130, 2, 2, 40, 72), (1, 300, 3, 1, 64, 200)], ids=str)
def test_every_row_head_and_chunk_as_the_plain_form(size, io):
    Case(*size, io).check(64)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 4200, 2, 1, 24, 40), (1, 4400, 1, 1, 72, 130), (2, 5121, 3, 3, 8, 8)], ids=str)
def test_every_chunk_of_long_rows_as_the_plain_form(size, io):
    """Rows that are cut into segments (the plain form by chunks alone: its steps would take minutes)."""
    Case(*size, io, decay=0.02).check(64, forms=(chunks,))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("up", [False, True], ids=["falling", "rising"])
def test_slopes_of_very_different_steps(up, io):
    """Slopes of 1 to 10^-7 within a chunk, eight steps of each size, later ones the smaller and the other way round."""
    sizes = 10.0 ** -(torch.arange(150) % 64 // 8).float()
    Case(2, 150, 2, 1, 24, 40, io, sizes=sizes.flip(0) if up else sizes).check(8, 2.0 ** -38)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_values_and_betas_of_very_different_sizes(io):
    Case(2, 150, 2, 1, 24, 40, io, columns=10.0 ** -(torch.arange(40) % 6).float()).check(64)
    Case(2, 150, 2, 1, 24, 40, io, betas=10.0 ** -(torch.arange(150) % 7).float()).check(64)


def test_slow_decays_over_many_chunks():
    """Nothing but decays (betas of 0) over 16384 steps: each of 256 chunks rounds its decay, a product and a sum.  Roundings of
    at most u that err to both sides alike have a root mean square of u / sqrt(3), so 768 of them add up to 16 u; five times that for
    the worst of 80 heads."""
    N, S, H, D = 40, 16384, 2, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    rate = torch.linspace(5e-5, 3e-4, N * H, device="cuda").view(N, 1, H)
    decay, state = -rate * (0.5 + r(N, S, H)), 1 + r(N, H, D, D)
    k, v = r(N, S, H, D), r(N, S, H, D)
    plan = orc.rnn_delta_create(H, D, D, layout=1)
    end = orc.delta_rule(plan, k, k, v, decay, torch.zeros_like(decay), None, state)[1]
    off = end.double() / (state.double() * decay.double().sum(1).exp()[..., None, None]) - 1
    assert float(off.mean((-1, -2)).abs().max()) <= 80 * U


def test_slow_decays_over_many_tokens():
    """The same a token at a time: 1500 tokens round a decay and a product each, 32 u; five times that for the worst of 64 heads."""
    N, S, H, D = 32, 1500, 2, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    decay, state = -(0.003 + 0.003 * r(S, N, H)), 1 + r(N, H, D, D)
    want = state.double() * decay.double().sum(0).exp()[..., None, None]
    plan, x, Y = orc.rnn_delta_create(H, D, D), r(N, H, D), torch.empty(N, H, D, device="cuda")
    beta = torch.zeros(N, H, device="cuda")
    for t in range(S):
        orc.rnn_delta_step(plan, x, x, x, decay[t], beta, state, Y)
    off = state.double() / want - 1
    assert float(off.mean((-1, -2)).abs().max()) <= 160 * U
