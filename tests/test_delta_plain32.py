"""The plain fp32 forms that the gated delta rule is compared with are its formulas, and the comparison catches operands
that have lost their second parts."""
import pytest
import torch

from delta_plain32 import chunks, groups, like_plain, plain_errors, steps


@pytest.fixture(autouse=True)
def one_thread():
    """Thousands of small operations: threads of several test processes would wait for one another."""
    threads = torch.get_num_threads()
    torch.set_num_threads(1)
    yield
    torch.set_num_threads(threads)


def _inputs(dY=1.0):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda t: 0.99 * t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    N, S, H, DK, DV = 1, 140, 2, 32, 24
    return [unit(r(N, S, H, DK)), unit(r(N, S, H, DK)), r(N, S, H, DV), -0.05 * torch.rand(N, S, H, generator=g),
            torch.rand(N, S, H, generator=g), r(N, H, DK, DV), dY * r(N, S, H, DV), 1e-9 * r(N, H, DK, DV), 0.2]


def _wide(ins):
    return [t.double() for t in ins[:-1]] + ins[-1:]


def test_chunks_are_the_steps():
    ins = _wide(_inputs())
    a, b = steps(*ins), chunks(*ins)
    assert set(a) == set(b)
    for name in a:
        assert torch.allclose(a[name], b[name], rtol=1e-10, atol=1e-12), name


def _check(got, want, plain, size=64, floor=0.0, names=None):
    for name in names or want:
        like_plain(name, groups(name, got[name].double(), size), groups(name, want[name], size), plain[name], 0.0, floor)


def test_operands_of_one_part_are_caught():
    ins = _inputs()
    want = steps(*_wide(ins))
    plain = plain_errors(ins, want, 64)
    _check(steps(*ins), want, plain)
    _check(chunks(*ins), want, plain)
    for i in range(3):      # Q, K or V without the second of its two fp16 parts
        one = list(ins)
        one[i] = ins[i].half().float()
        with pytest.raises(AssertionError):
            _check(steps(*one), want, plain)


def test_a_small_step_that_is_lost_is_caught():
    ins = _inputs((10.0 ** -(torch.arange(140) % 64 // 8).float())[None, :, None, None])
    want = steps(*_wide(ins))
    plain = plain_errors(ins, want, 8)
    _check(steps(*ins), want, plain, 8, 2.0 ** -38)
    # dY to a multiple of 2^-25 of its chunk's largest
    step, lost = 2.0 ** -25 * float(ins[6].abs().max()), list(ins)
    lost[6] = (ins[6] / step).round() * step
    with pytest.raises(AssertionError):
        _check(steps(*lost), want, plain, 8, 2.0 ** -38, ("dQ",))
