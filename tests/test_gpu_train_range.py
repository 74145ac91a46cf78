"""Gradients whose value is in range although a product of two of their factors is not."""
import pytest
import torch

from tests.test_gpu_train import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kept", ["act", "8bit"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,I,k", [(20, 128, 3, 32, 1), (64, 2560, 1, 640, 1), (300, 128, 2, 288, 2)])
def test_large_factors_and_a_closed_gate(T, H, E, I, k, act, kept):
    """dh u = 1e42 is past float32, and dg = dh u silu'(-60) = -5e17 is not.  At g = -100 the
    slope itself is past float32's range, on the other side: dg is held to be finite."""
    c = Case(T, H, E, I, k, act, kept, seed=41)
    c.dy.zero_()
    c.dy[:, 0] = 1e22
    c.w[2].zero_()
    c.w[2][:, 0, :] = 1.0
    c.u.fill_(1e20)
    c.g.fill_(-60.0)
    c.fill_saved()
    c.backward()
    c.check_backward(f"large factors {T} {H} {E} {I} {act} {kept}")
    c.g.fill_(-100.0)
    if kept == "act":
        c.g_out.t.copy_(c.g)
        c.backward()
        assert all(bool(torch.isfinite(v).all()) for v in c.grads().values())


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_small_and_a_large_factor(act):
    """The other way round: u silu'(-60) = 5e-45 has lost its digits, dh u has not."""
    c = Case(40, 128, 2, 64, 1, act, seed=42)
    c.dy.zero_()
    c.dy[:, 0] = 1e30
    c.w[2].zero_()
    c.w[2][:, 0, :] = 1.0
    c.u.fill_(1e-20)
    c.g.fill_(-60.0)
    c.fill_saved()
    c.backward()
    c.check_backward(f"small and large factor {act}")
    c.dy[:, 0] = 1e-20
    c.u.fill_(1e30)
    c.fill_saved()
    c.backward()
    c.check_backward(f"large and small factor {act}")
