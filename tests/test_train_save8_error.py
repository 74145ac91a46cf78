"""The error of 8-bit checkpoints that the header states, on the 64-bit definition
that the kernels are held to bit for bit (no GPU needed)."""
import pytest
import torch

from tests import train_ref as R


def error(v):
    """Scale, unit, error and largest magnitude of each 32 elements."""
    v = v.double().reshape(-1, 32)
    s = R.scales8(v)
    back = R.values8(R.codes8(v, s), s)
    return s[:, 0].long(), R.pow2(s[:, 0].long() - 127), (back - v).abs().amax(1), v.abs().amax(1)


def groups(dtype, exponents):
    """32 elements each whose largest magnitude is around 2^e."""
    g = torch.Generator().manual_seed(1)
    e = torch.tensor(exponents, dtype=torch.float64)[:, None, None]
    v = (torch.rand(1, 200, 32, generator=g, dtype=torch.float64) * 2 - 1) * torch.exp2(e)
    v[:, :, 3] = torch.exp2(e[:, :, 0]) * torch.linspace(0.5, 1, 200, dtype=torch.float64)
    big = torch.finfo(dtype).max
    return v.clamp(-big, big).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_error_of_a_checkpoint(dtype):
    s, unit, err, top = error(groups(dtype, [-140, -133, -130, -127, -126, -121, -119, -118, -60, -1, 0, 1, 40, 120, 127, 128]))
    assert bool((s == 1).any()) and bool((s == 248).any()) and int(s.max()) == 248
    cut = (s == 248) & (top > 127 * unit)
    assert bool((err[~cut] <= unit[~cut] / 2).all()) and bool((err < unit).all())
    assert bool((err[s > 1] * 127 <= top[s > 1]).all())
    assert bool((err[s == 1] <= 2.0 ** -127).all())


def test_where_half_a_unit_and_1_127_do_not_hold():
    """The largest float32 numbers lose nearly a unit, the smallest all they have."""
    v = torch.zeros(2, 32)
    v[0, 0], v[1, 0] = torch.finfo(torch.float32).max, 2.0 ** -130
    s, unit, err, top = error(v)
    assert s.tolist() == [248, 1]
    assert float(err[0]) > 0.99 * float(unit[0]) and float(err[1]) == float(top[1])
    v = torch.zeros(1, 32, dtype=torch.bfloat16)
    v[0, 0] = torch.finfo(torch.bfloat16).max
    s, unit, err, top = error(v)
    assert s.tolist() == [248] and float(err[0]) == float(unit[0]) / 2
