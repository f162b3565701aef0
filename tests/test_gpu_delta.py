"""The gated delta rule on the GPU against its formula in 64 bits: runs, gradients and single tokens over types,
head layouts, odd sizes, lengths, strides and streams."""
import pytest
import torch

import delta_ref64 as ref
import onnx_recurrent_gb300 as orc

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """A plan and inputs on the GPU with their 64-bit copies in layout 1 on the CPU."""

    def __init__(self, N, S, H, HK, DK, DV, io="f32", layout=1, lens=None, carried=False, wide=False, seed=0, decay=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        unit = lambda t: 0.99 * t / t.norm(dim=-1, keepdim=True)     # noqa: E731  (below 1 after any rounding)
        self.N, self.S, self.io, self.layout, self.terms = N, S, io, layout, DK + 128
        self.plan = orc.rnn_delta_create(H, key_size=DK, value_size=DV, key_heads=HK, layout=layout, scale=scale)
        orc.rnn_delta_set_io_type(self.plan, io)
        dt = DT[io]
        cpu = [unit(r(N, S, HK, DK)).to(dt), unit(r(N, S, HK, DK)).to(dt), r(N, S, H, DV).to(dt),
               -decay * torch.rand(N, S, H, generator=g), torch.rand(N, S, H, generator=g)]
        self.dY = r(N, S, H, DV).to(dt)
        self.wide = wide
        self.gpu, self.dYg = [self.put(t) for t in cpu], self.put(self.dY)
        self.ref = [t.double() for t in cpu]
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
        self.glens = None if lens is None else self.lens.cuda()
        self.state = r(N, H, DK, DV) if carried else None
        self.d_state = r(N, H, DK, DV) if carried else None
        self.gstate, self.gd_state = (None if t is None else t.cuda() for t in (self.state, self.d_state))
        up = lambda t: None if t is None else t.double()  # noqa: E731
        self.want = ref.delta(*self.ref, self.lens, up(self.state), self.plan.scale)
        self.grads = lambda: ref.delta_grad(self.dY.double(), up(self.d_state), *self.ref, self.lens, up(self.state), self.plan.scale)

    def put(self, t):
        t = (t if self.layout == 1 else t.transpose(0, 1)).contiguous().cuda()
        if self.wide:       # a part of a wider tensor, one element off
            flat = t.flatten(2)
            w = torch.full((*flat.shape[:2], flat.shape[2] + 7), float("nan"), dtype=t.dtype, device="cuda")
            w[..., 1:1 + flat.shape[2]] = flat
            return w[..., 1:1 + flat.shape[2]].unflatten(2, t.shape[2:])
        return t

    def back(self, t):
        return t if self.layout == 1 else t.transpose(0, 1)

    def check(self, what="", u=ref.U):
        Y, state, saved = orc.delta_rule(self.plan, *self.gpu, self.glens, self.gstate, save=True)
        ref.close(self.back(Y), self.want[0], self.S, self.terms, self.io, what + "Y", u)
        ref.close(state, self.want[1], self.S, self.terms, "f32", what + "state", u)
        out = orc.delta_rule_grad(self.plan, self.dYg, saved, *self.gpu, self.glens, self.gstate, d_state=self.gd_state)
        orc.rnn_delta_sync(self.plan)
        want = self.grads()
        assert set(out) == set(want)
        for name, t in out.items():
            io = self.io if name in ("dQ", "dK", "dV") else "f32"
            # dQ, dK and dg are sums of DV (dg of DK DV) products of two run results, each off by the run's error
            ref.close(t if name == "d_initial_state" else self.back(t), want[name], 3 * self.S,
                      self.terms + self.plan.value_size, io, what + name, u)
        return Y, state, out


# one step, a chunk less, exactly and more than one, several; heads that share keys; sizes of no multiple
SIZES = [(1, 1, 1, 1, 1, 1), (2, 63, 2, 1, 8, 16), (1, 64, 2, 2, 16, 32), (2, 65, 3, 3, 20, 33), (1, 130, 4, 2, 64, 64),
         (3, 100, 6, 2, 40, 72), (1, 200, 1, 1, 128, 128), (2, 129, 2, 1, 127, 161), (1, 70, 2, 2, 96, 200)]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_run_and_gradient(size, io):
    Case(*size, io=io, layout=size[1] % 2, carried=size[0] > 1).check()


# few heads and long rows, whose chain is cut into segments: whole ones, ragged ones, a last one of a few steps
LONG = [(1, 4096, 1, 1, 16, 32), (2, 4200, 2, 1, 20, 40), (1, 4400, 1, 1, 72, 130), (1, 5121, 3, 3, 8, 8)]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", LONG, ids=str)
def test_long_rows(size, io):
    c = Case(*size, io=io, carried=True, decay=0.3)
    c.check()
    assert orc.rnn_delta_last_launch_count(c.plan) == 2        # the gradient's
    orc.delta_rule(c.plan, *c.gpu)
    assert orc.rnn_delta_last_launch_count(c.plan) == 4


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_rows_of_other_lengths_in_place(io):
    lens = [4500, 0, 3, 2700, 64]
    c = Case(5, 4500, 2, 1, 24, 48, io=io, layout=0, lens=lens, carried=True, decay=0.3)
    Y, state, _ = c.check()
    st, y = c.gstate.clone(), torch.full_like(Y, 7.0)
    orc.rnn_delta_rule(c.plan, *c.gpu, c.glens, st, y, st)
    assert torch.equal(st, state) and torch.equal(y, Y)
    # without a state to begin with, as with zeros
    a = orc.delta_rule(c.plan, *c.gpu, c.glens)
    b = orc.delta_rule(c.plan, *c.gpu, c.glens, torch.zeros_like(st))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rows_of_other_lengths(io):
    c = Case(6, 150, 2, 1, 32, 48, io=io, lens=[150, 0, 1, 64, 65, 149], carried=True)
    Y, state, out = c.check()
    for n, ln in enumerate([150, 0, 1, 64, 65, 149]):
        assert not Y[n, ln:].any()
        for name in ("dQ", "dK", "dV", "dg", "dbeta"):
            assert not out[name][n, ln:].any(), (name, n)
    assert torch.equal(state[1], c.gstate[1]) and torch.equal(out["d_initial_state"][1], c.gd_state[1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
def test_parts_of_wider_tensors(io, layout):
    Case(2, 90, 2, 2, 24, 40, io=io, layout=layout, wide=True).check()


def test_outputs_into_parts_of_wider_tensors_leave_the_rest():
    c = Case(2, 70, 2, 1, 16, 24, lens=[70, 20])
    big = torch.full((2, 70, 3 * 48), 7.0, device="cuda")
    Y = big[..., 48:96].unflatten(-1, (2, 24))
    orc.rnn_delta_rule(c.plan, *c.gpu, c.glens, None, Y)
    ref.close(Y, c.want[0], 70, c.terms, "f32", "Y")
    assert (big[..., :48] == 7).all() and (big[..., 96:] == 7).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_and_no_decay(io):
    Case(1, 140, 2, 2, 16, 32, io=io, decay=0.0).check("none ")
    Case(1, 140, 2, 2, 16, 32, io=io, decay=60.0).check("strong ")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_state_that_is_forgotten(io):
    """g of -inf or of a type's lowest value: the steps after it are those of a state of zeros."""
    c = Case(1, 120, 1, 1, 16, 16, io=io, carried=True)
    for at, v in ((30, float("-inf")), (64, torch.finfo(torch.float32).min), (100, -2000.0)):
        c.gpu[3][0, at], c.ref[3][0, at] = v, -1e4
    c.want = ref.delta(*c.ref, None, c.state.double(), c.plan.scale)
    c.check()


def test_nan_stays_in_its_head_and_row():
    c = Case(2, 80, 2, 2, 16, 16, carried=True)
    c.gpu[2][0, 10, 1, 3] = float("nan")
    Y, state, _ = orc.delta_rule(c.plan, *c.gpu, None, c.gstate)
    assert Y[0, 10:, 1, 3].isnan().all() and not Y[0, :, 0].isnan().any() and not Y[1].isnan().any()
    assert not state[1].isnan().any() and state[0, 1].isnan().any()


def test_lengths_out_of_range_are_clamped_and_reported():
    c = Case(3, 70, 1, 1, 8, 8)
    bad = torch.tensor([70, 71, -1], dtype=torch.int32, device="cuda")
    Y, state, _ = orc.delta_rule(c.plan, *c.gpu, bad)
    with pytest.raises(orc.RNNError):
        orc.rnn_delta_sync(c.plan)
    orc.rnn_delta_sync(c.plan)
    ref.close(Y[:2], c.want[0][:2], 70, c.terms, "f32", "Y")
    assert not Y[2].any() and not state[2].any()


def test_nothing_to_run():
    p = orc.rnn_delta_create(2, 8, 8, layout=1)
    t = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    st = torch.randn(2, 2, 8, 8, device="cuda")
    Y, end, saved = orc.delta_rule(p, t(2, 0, 2, 8), t(2, 0, 2, 8), t(2, 0, 2, 8), t(2, 0, 2), t(2, 0, 2), None, st, save=True)
    assert Y.shape == (2, 0, 2, 8) and torch.equal(end, st) and saved.numel() == 0
    out = orc.delta_rule_grad(p, Y, saved, t(2, 0, 2, 8), t(2, 0, 2, 8), t(2, 0, 2, 8), t(2, 0, 2), t(2, 0, 2), None, st, st)
    assert torch.equal(out["d_initial_state"], st)
    Y, end, _ = orc.delta_rule(p, t(0, 5, 2, 8), t(0, 5, 2, 8), t(0, 5, 2, 8), t(0, 5, 2), t(0, 5, 2))
    assert Y.shape == (0, 5, 2, 8) and end.shape == (0, 2, 8, 8)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_states_in_place(io):
    c = Case(2, 140, 2, 1, 32, 64, io=io, carried=True)
    st, Y = c.gstate.clone(), torch.empty(2, 140, 2, 64, device="cuda", dtype=DT[io])
    orc.rnn_delta_rule(c.plan, *c.gpu, None, st, Y, st)
    want = orc.delta_rule(c.plan, *c.gpu, None, c.gstate, save=True)
    assert torch.equal(st, want[1]) and torch.equal(Y, want[0])
    g = c.gd_state.clone()
    orc.rnn_delta_rule_grad(c.plan, c.dYg, want[2], *c.gpu, None, g, d_initial_state=g)
    full = orc.delta_rule_grad(c.plan, c.dYg, want[2], *c.gpu, None, c.gstate, c.gd_state)
    assert torch.equal(g, full["d_initial_state"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_each_gradient_alone_and_twice_the_same(io):
    c = Case(2, 130, 4, 2, 32, 48, io=io, carried=True)
    _, _, saved = orc.delta_rule(c.plan, *c.gpu, None, c.gstate, save=True)
    full = orc.delta_rule_grad(c.plan, c.dYg, saved, *c.gpu, None, c.gstate, c.gd_state)
    for name, t in full.items():
        one = torch.empty_like(t)
        orc.rnn_delta_rule_grad(c.plan, c.dYg, saved, *c.gpu, None, c.gd_state, **{name: one})
        assert torch.equal(one, t), name


def test_gradient_against_differences_of_the_run():
    """Central differences of the run itself in fp32: a step e errs by the run's own error over e."""
    c = Case(1, 70, 2, 1, 8, 8, carried=True, decay=0.2)
    args = [*c.gpu, c.gstate]
    _, _, saved = orc.delta_rule(c.plan, *c.gpu, None, c.gstate, save=True)
    out = orc.delta_rule_grad(c.plan, c.dYg, saved, *c.gpu, None, c.gstate, c.gd_state)
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, name in enumerate(["dQ", "dK", "dV", "dg", "dbeta", "d_initial_state"]):
        way = torch.randn(args[i].shape, generator=g, device="cuda")
        way /= way.norm()

        def loss(step):
            a = list(args)
            a[i] = a[i] + step * way
            Y, end, _ = orc.delta_rule(c.plan, *a[:5], None, a[5])
            return float((Y.double() * c.dYg.double()).sum() + (end.double() * c.gd_state.double()).sum())
        e = 0.02
        # five points: what is left of the fourth order, and the runs' error of about 10^-5 over the step
        slope = (8 * (loss(e) - loss(-e)) - (loss(2 * e) - loss(-2 * e))) / (12 * e)
        got = float((out[name].double() * way.double()).sum())
        assert abs(got - slope) < 2e-3 * max(1.0, float(out[name].norm())), (name, got, slope)


def test_a_prompt_in_two_parts_and_tokens():
    """A prompt, its continuation from the carried state and single tokens give what one run gives."""
    c = Case(3, 140, 4, 2, 32, 40, io="bf16")
    first, second = ([t[:, :77] for t in c.gpu], [t[:, 77:130] for t in c.gpu])
    _, st, _ = orc.delta_rule(c.plan, *first)
    Y2, st, _ = orc.delta_rule(c.plan, *second, None, st)
    ref.close(Y2, c.want[0][:, 77:130], 140, c.terms, "bf16", "Y")
    for t in range(130, 140):
        y = torch.empty(3, 4, 40, device="cuda", dtype=torch.bfloat16)
        orc.rnn_delta_step(c.plan, *(v[:, t] for v in c.gpu), st, y)
        ref.close(y, c.want[0][:, t], 140, c.terms, "bf16", f"token {t}")
    ref.close(st, c.want[1], 140, c.terms, "f32", "state")


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (5, 2, 1, 20, 33), (3, 4, 4, 64, 64), (7, 3, 1, 128, 200), (2, 2, 2, 127, 128)], ids=str)
def test_single_tokens(size, io):
    N, H, HK, DK, DV = size
    c = Case(N, 1, H, HK, DK, DV, io=io, carried=True, wide=N > 3)
    one = [t[:, 0] for t in c.gpu]
    out, Y = torch.empty_like(c.gstate), torch.empty(N, H, DV, device="cuda", dtype=DT[io])
    orc.rnn_delta_step(c.plan, *one, c.gstate, Y, state_out=out)
    ref.close(Y, c.want[0][:, 0], 1, c.terms, io, "Y")
    ref.close(out, c.want[1], 1, c.terms, "f32", "state")
    orc.rnn_delta_step(c.plan, *one, c.gstate, Y)
    assert torch.equal(c.gstate, out)


def test_slots():
    c = Case(4, 1, 2, 1, 24, 36, carried=True)
    table = torch.full((6, 2, 24, 36), 9.0, device="cuda")
    table[5], table[0], table[3] = c.gstate[0], c.gstate[1], c.gstate[3]
    slots = torch.tensor([5, 0, -1, 3], dtype=torch.int32, device="cuda")
    Y = torch.full((4, 2, 36), 5.0, device="cuda")
    one = [t[:, 0] for t in c.gpu]
    orc.rnn_delta_step(c.plan, *one, table, Y, slots=slots)
    orc.rnn_delta_sync(c.plan)
    for n, s in ((0, 5), (1, 0), (3, 3)):
        ref.close(table[s], c.want[1][n], 1, c.terms, "f32", "state")
        ref.close(Y[n], c.want[0][n, 0], 1, c.terms, "f32", "Y")
    assert not Y[2].any() and (table[[1, 2, 4]] == 9).all()
    before = table.clone()
    orc.rnn_delta_step(c.plan, *one, table, Y, slots=torch.tensor([6, -1, -2, -1], dtype=torch.int32, device="cuda"))
    with pytest.raises(orc.RNNError):
        orc.rnn_delta_sync(c.plan)
    assert torch.equal(table, before) and not Y.any()


def test_captured_calls_and_another_stream():
    c = Case(2, 130, 2, 2, 32, 32, io="bf16", carried=True)
    want = orc.delta_rule(c.plan, *c.gpu, None, c.gstate, save=True)
    grads = orc.delta_rule_grad(c.plan, c.dYg, want[2], *c.gpu, None, c.gstate, c.gd_state)
    plan = orc.rnn_delta_create(2, 32, 32, layout=1)
    orc.rnn_delta_set_io_type(plan, "bf16")
    Y, st, saved = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(want[2])
    out = {n: torch.empty_like(t) for n, t in grads.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):       # the plan's first calls
        orc.rnn_delta_rule(plan, *c.gpu, None, c.gstate, Y, st, saved)
        orc.rnn_delta_rule_grad(plan, c.dYg, saved, *c.gpu, None, c.gd_state, **out)
    for _ in range(2):
        for t in (Y, st, saved, *out.values()):
            t.zero_()
        graph.replay()
        orc.delta_rule(plan, *[torch.cat([t, t], 1) for t in c.gpu])       # a larger plain call beside it
        torch.cuda.synchronize()
        assert torch.equal(Y, want[0]) and torch.equal(st, want[1])
        assert all(torch.equal(out[n], grads[n]) for n in grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y2, st2, saved2 = orc.delta_rule(plan, *c.gpu, None, c.gstate, save=True, stream=side)
    out2 = orc.delta_rule_grad(plan, c.dYg, saved2, *c.gpu, None, c.gstate, c.gd_state, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(Y2, want[0]) and torch.equal(st2, want[1]) and all(torch.equal(out2[n], grads[n]) for n in grads)
