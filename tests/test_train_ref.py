"""The 64-bit definitions that the training kernels are tested against: the
gradients against differences of the products they belong to, the checkpoints
at the borders of their scales (CPU)."""
import math

import pytest
import torch

from tests import train_ref as R


def _routes(T, Ex, k, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(Ex, generator=g)[:k] for _ in range(T)])
    expert = ids.reshape(-1).clone()
    expert[torch.rand(T * k, generator=g) < drop] = Ex
    order = torch.argsort(expert, stable=True)
    offsets = torch.zeros(Ex + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(torch.bincount(expert, minlength=Ex + 1)[:Ex], 0)
    pair = torch.full((T * k,), -1, dtype=torch.int64)
    n = int(offsets[Ex])
    pair[:n] = order[:n]
    return ids, offsets, pair


def test_gradients_are_those_of_differences():
    T, H, Ex, I, k = 5, 6, 4, 3, 2
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    ids, offsets, pair = _routes(T, Ex, k, 2, 0.2)
    n = int(offsets[Ex])
    x, wg, wu, wd, dy = rnd(T, H), rnd(Ex, I, H), rnd(Ex, I, H), rnd(Ex, H, I), rnd(T * k, H)

    def loss(rows, wg, wu, wd):
        """sum of dy * y with each row its own input."""
        total = 0.0
        for e in range(Ex):
            a, b, _ = R.rows_of(offsets, pair, k, e)
            g, u = rows[a:b] @ wg[e].t(), rows[a:b] @ wu[e].t()
            total += float((dy[a:b] * ((g / (1 + torch.exp(-g)) * u) @ wd[e].t())).sum())
        return total

    rows = torch.zeros(T * k, H, dtype=torch.float64)
    rows[:n] = x[pair[:n] // k]
    fwd = R.gate_up(x, wg, wu, offsets, pair, k, torch.float64)
    got = R.backward(dy, x, fwd["g"][0], fwd["u"][0], wg, wu, wd, offsets, pair, k, torch.float64)
    at = dict(drows=rows, dgate=wg, dup=wu, ddown=wd)
    eps = 1e-6
    for name, t in at.items():
        for i in range(t.numel() if name != "drows" else n * H):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[i] = eps
            args = lambda s: [at[m] + (s * d.reshape(t.shape) if m == name else 0) for m in at]
            diff = (loss(*args(1)) - loss(*args(-1))) / (2 * eps)
            assert math.isclose(diff, float(got[name][0].reshape(-1)[i]), rel_tol=1e-6, abs_tol=1e-7), (name, i)


def test_router_gradient_is_that_of_differences():
    T, H, Ex, k = 3, 4, 6, 3
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, wr, bias, dw = rnd(T, H), rnd(Ex, H), rnd(Ex), rnd(T, k)
    ids = (x @ wr.t() + bias).topk(k, dim=1).indices

    def weights(x, wr, bias):
        return torch.softmax((x @ wr.t() + bias).gather(1, ids), dim=1)

    got = R.router(ids, weights(x, wr, bias), dw, x, wr, None, torch.float64)
    at, eps = dict(dx=x, dw_router=wr, dbias=bias), 1e-6
    for name, t in at.items():
        for i in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[i] = eps
            f = lambda s: float((dw * weights(*[at[m] + (s * d.reshape(t.shape) if m == name else 0) for m in at])).sum())
            diff = (f(1) - f(-1)) / (2 * eps)
            assert math.isclose(diff, float(got[name][0].reshape(-1)[i]), rel_tol=1e-6, abs_tol=1e-8), (name, i)


@pytest.mark.parametrize("top,scale", [
    (0.0, 1), (2.0 ** -140, 1), (127.0, 127), (127.5, 128), (1.0, 121), (1.984375, 121), (1.9921875, 122),
    (2.0, 122), (3.0e38, 248), (3.4e38, 248), (float("inf"), 255), (float("nan"), 255), (127 * 2.0 ** -126, 1),
    (128 * 2.0 ** -126, 2)])
def test_scales(top, scale):
    v = torch.zeros(1, 64, dtype=torch.float64)
    v[0, 40], v[0, 3] = -top, 2.0
    s = R.scales8(v)
    assert s.tolist() == [[122, scale]]
    back = R.values8(R.codes8(v, s), s)
    if scale == 255:
        assert bool(torch.isnan(back[0, 32:]).all()) and back[0, 3] == 2.0
    else:
        # half a unit; past 127 units of the largest scale the code is cut
        assert float((back - v).abs().max()) <= max(2.0 ** (scale - 128), top - 127 * 2.0 ** (scale - 127))
        assert float(back.abs().max()) <= torch.finfo(torch.bfloat16).max
