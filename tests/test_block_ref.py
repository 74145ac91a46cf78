"""The 64-bit definitions that the GPU tests of the operators around the
routed experts compare with: their gradients against central differences and
against torch's own differentiation of the forward formulas (CPU)."""
import pytest
import torch

from tests import block_ref as R

EPS = 1e-5


def _normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _difference(f, t, h=1e-5):
    g = torch.empty_like(t)
    for i in range(t.numel()):
        old = t.reshape(-1)[i].item()
        t.reshape(-1)[i] = old + h
        up = f().item()
        t.reshape(-1)[i] = old - h
        down = f().item()
        t.reshape(-1)[i] = old
        g.reshape(-1)[i] = (up - down) / (2 * h)
    return g


FLAGS = [0, R.GATE_TOKEN, R.GATE_FULL, R.GATE_TOKEN | R.SIGMOID, R.GATE_FULL | R.SIGMOID, R.NO_NORM,
         R.NO_NORM | R.GATE_FULL | R.SIGMOID, R.NO_NORM | R.GATE_TOKEN]


@pytest.mark.parametrize("flags", FLAGS)
def test_norm_gradient_is_the_difference(flags):
    T, H = 3, 5
    z, w, res, dout = (_normal(T, H, seed=1), _normal(H, seed=2), _normal(T, H, seed=3),
                       _normal(T, H, seed=4))
    gate = None
    if flags & (R.GATE_TOKEN | R.GATE_FULL):
        gate = _normal(*((T,) if flags & R.GATE_TOKEN else (T, H)), seed=5)
    kw = dict(dtype=torch.float64, eps=EPS, offset=1.0, rscale=0.5, bscale=0.7, flags=flags)

    def loss():
        v = R.norm_out(z, torch.zeros_like(z), w, gate, res, None, **kw)["out"][0]
        return (v * dout).sum()

    g = R.norm_bwd(dout, z, w, gate, None, **kw)
    # truncation h^2 ~ 1e-10 and cancellation 2^-53 / h ~ 1e-11, times small factors
    assert (g["dz"][0] - _difference(loss, z)).abs().max() < 1e-7
    if not flags & R.NO_NORM:
        assert (g["dw"][0] - _difference(loss, w)).abs().max() < 1e-7
    if gate is not None:
        assert (g["dgate"][0] - _difference(loss, gate)).abs().max() < 1e-7


def test_next_norm_and_residual_gradient_chain():
    """Gradient of out and n_next together: moe_norm_in_backward of the next
    norm with dres, then moe_norm_out_backward, as include/moe.h states."""
    T, H = 4, 6
    z, w, res, wn = _normal(T, H, seed=1), _normal(H, seed=2), _normal(T, H, seed=3), _normal(H, seed=4)
    d_out, d_next = _normal(T, H, seed=5), _normal(T, H, seed=6)
    kw = dict(dtype=torch.float64, eps=EPS, offset=0.0, rscale=0.5, bscale=0.7, flags=0)
    leaves = [t.clone().requires_grad_() for t in (z, w, res, wn)]
    o = R.norm_out(leaves[0], torch.zeros_like(z), leaves[1], None, leaves[2], leaves[3], **kw)
    ((o["out"][0] * d_out).sum() + (o["n_next"][0] * d_next).sum()).backward()
    v = o["out"][0].detach()
    nxt = R.norm_bwd(d_next, v, wn, None, d_out, **{**kw, "rscale": 1.0, "bscale": 1.0})
    own = R.norm_bwd(nxt["dz"][0], z, w, None, None, **kw)
    assert (own["dz"][0] - leaves[0].grad).abs().max() < 1e-12
    assert (own["dw"][0] - leaves[1].grad).abs().max() < 1e-12
    assert (0.5 * nxt["dz"][0] - leaves[2].grad).abs().max() < 1e-12
    assert (nxt["dw"][0] - leaves[3].grad).abs().max() < 1e-12


def _pairs(T, k, E, drop, seed):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g, dtype=torch.float64)
    top, ids = logits.topk(k, dim=1)
    order = ids.reshape(-1).argsort(stable=True)
    row = torch.empty(T * k, dtype=torch.int64)
    row[order] = torch.arange(T * k)
    if drop:
        row[torch.rand(T * k, generator=g) < drop] = -1
    return logits, ids, torch.softmax(top, 1), row.to(torch.int32)


@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_dispatch_and_combine_gradients_are_differences(drop):
    T, k, E, H = 4, 2, 5, 3
    _, _, w, row = _pairs(T, k, E, drop, 0)
    x, y, drows, dout = (_normal(T, H, seed=1), _normal(T * k, H, seed=2), _normal(T * k, H, seed=3),
                         _normal(T, H, seed=4))
    zero = torch.zeros(T * k, H, dtype=torch.float64)
    kw = dict(dtype=torch.float64)
    g = R.dispatch_bwd(drows, row, w, x, None, T, dw=True, **kw)
    loss = lambda: (R.dispatch(x, row, w, zero, **kw)["rows"][0] * drows).sum()
    assert (g["dx"][0] - _difference(loss, x)).abs().max() < 1e-8
    assert (g["dw"][0] - _difference(loss, w)).abs().max() < 1e-8
    g = R.combine_bwd(dout, y, row, w, zero, dw=True, **kw)
    loss = lambda: (R.combine(y, row, w, T, k)[0] * dout).sum()
    assert (g["dy"][0] - _difference(loss, y)).abs().max() < 1e-8
    assert (g["dw"][0] - _difference(loss, w)).abs().max() < 1e-8


def test_route_gradient_is_the_difference():
    T, k, E = 3, 3, 7
    logits, ids, w, _ = _pairs(T, k, E, 0.0, 1)
    dw = _normal(T, k, seed=2)
    loss = lambda: (torch.softmax(logits.gather(1, ids), 1) * dw).sum()
    want = _difference(loss, logits)
    got = R.route_bwd(ids, w, dw, E)["dlogits"][0]
    assert (got - want).abs().max() < 1e-8
