"""Gradient of a sigmoid gate over the whole range of the gate, on the GPU
against 64-bit definitions.

With e = exp(-|g|) the slope is e / (1 + e)^2 on both sides of 0; none of its
steps cancels.  Counted in units of 2^-24 of the slope: the exponential 4 and
2.5 |g| where its argument is a rounded product g log2(e) (the product and the
constant are off by 2^-24 and 2^-26 of an argument of 1.45 |g|), the sum 1, the
reciprocal 2, the products of e r (1 - e r) 4, each use of e and r counted
once more: 24 + 2.5 |g|."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests import block_ref as R
from tests.test_gpu_block import DEV, DT, EPS, FULL, NONORM, SIG, TOKEN, Gen, Out, workspace

pytestmark = pytest.mark.gpu

POINTS = [0.0, 15.0, -15.0, 10.0, 12.0, -12.0, 17.0, -17.0, 20.0, 30.0, -30.0, -0.0, 88.0, -88.0, 104.0, -104.0]


def gates(g, *shape, dtype):
    """The points first, the rest evenly over +-30, in an order of its own."""
    n = 1
    for s in shape:
        n *= s
    v = torch.linspace(-30, 30, n, device=DEV)[torch.randperm(n, generator=g.g, device=DEV)]
    m = min(n, len(POINTS))
    v[:m] = torch.tensor(POINTS[1:] + POINTS[:1], device=DEV)[:m]
    return v.view(*shape).to(dtype)


def gate_gradient(dout, z, w, gate, *, eps, bscale, flags, dtype):
    """(dgate, bound) of dz's gate."""
    z, T, H = z.double(), z.shape[0], z.shape[1]
    raw = gate.double().reshape(T, -1)
    e = torch.exp(-raw.abs())
    slope, rel = e / (1 + e) ** 2, (24 + 2.5 * raw.abs()) * R.E
    b = z
    if not flags & NONORM:
        b = z * ((z * z).mean(1, keepdim=True) + eps) ** -0.5 * w.double()
        rel = rel + (R.chain(H) / 2 + 4) * R.E
    t = bscale * dout.double() * b * slope
    if flags & TOKEN:
        return t.sum(1), (t.abs() * ((R.chain(H) + 14) * R.E + rel)).sum(1) + R.TINY * H
    return t, t.abs() * (10 * R.E + rel + R.u_of(dtype)) + R.TINY


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [TOKEN | SIG, FULL | SIG, TOKEN | SIG | NONORM, FULL | SIG | NONORM])
@pytest.mark.parametrize("T,H", [(1, 2560), (5, 77), (40, 2560), (17, 9000), (3, 40000), (2051, 1280), (2050, 40),
                                 (2051, 129), (16391, 333), (4, 1)])
def test_sigmoid_gate_gradient(T, H, flags, act):
    dt, g = DT[act], Gen(T, H, flags, act == "f32", 41)
    z, dout = g(T, H, dtype=dt), g(T, H, std=0.5, dtype=dt)
    w = None if flags & NONORM else g(H, std=0.2, mean=1.0, dtype=dt)
    gate = gates(g, T, dtype=torch.float32) if flags & TOKEN else gates(g, T, H, dtype=dt)
    norm = M.make_norm(T, H, act, eps=EPS, branch_scale=1.25, flags=flags)
    ws, nb = workspace(norm)
    dz, dg = Out(T, H, dtype=dt), Out(*gate.shape, dtype=gate.dtype)
    dw = Out(H, dtype=torch.float32) if w is not None else None
    M.moe_norm_out_backward(norm, dout, z, w, gate, dz.t, dg.t, dw.t if dw else None, ws, nb)
    want = {"dgate": gate_gradient(dout, z, w, gate, eps=EPS, bscale=1.25, flags=flags, dtype=gate.dtype)}
    R.check({"dgate": dg.t}, want, f"sigmoid gate {T}x{H} {act} {flags}")
    full = R.norm_bwd(dout, z, w, gate, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.25, flags=flags)
    R.check({"dz": dz.t}, {"dz": full["dz"]}, "dz")
    assert dz.ok() and dg.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [TOKEN, FULL])
@pytest.mark.parametrize("T,H", [(4, 96), (4, 40000), (2052, 96), (2052, 2560)])
def test_gate_at_infinity(T, H, kind, act):
    """sigmoid is 1 or 0 there, its slope 0."""
    dt, g = DT[act], Gen(T, H, kind, 43)
    z, dout = g(T, H, dtype=dt), g(T, H, dtype=dt)
    gate = g(T) if kind == TOKEN else g(T, H, dtype=dt)
    gate[0], gate[1] = float("inf"), -float("inf")
    norm = M.make_norm(T, H, act, flags=kind | SIG | NONORM)
    dz, dg = Out(T, H, dtype=dt), Out(*gate.shape, dtype=gate.dtype)
    M.moe_norm_out_backward(norm, dout, z, None, gate, dz.t, dg.t, None, None, 0)
    assert (dg.t[:2] == 0).all() and torch.equal(dz.t[0], dout[0]) and (dz.t[1] == 0).all()
    assert dg.t.isfinite().all() and dz.t.isfinite().all() and dz.ok() and dg.ok()
