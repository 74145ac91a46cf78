"""tests/train_layer_ref.py itself: its gradient against torch's differentiation in
float64, and that its bounds notice mistakes (no GPU needed)."""
import pytest
import torch

from tests.train_layer_ref import layer

CASES = [(20, 256, 6, 96, 3), (60, 128, 4, 64, 2), (7, 128, 16, 32, 5)]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(T, H, E, I, k, act="bf16"):
    g = torch.Generator().manual_seed(T + H)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DT[act])
    x, wr, w = r(T, H), r(E, H, std=0.05), [r(E, *s, std=0.05) for s in ((I, H), (I, H), (H, I))]
    bias = torch.randn(E, generator=g) * 0.1
    ids = torch.topk(x.double() @ wr.double().t() + bias.double(), k, dim=1)[1]
    return dict(x=x, wr=wr, bias=bias, w=w, ids=ids, residual=x, dout=r(T, H), dx_in=r(T, H))


@pytest.mark.parametrize("T,H,E,I,k", CASES)
def test_against_autograd(T, H, E, I, k):
    a = inputs(T, H, E, I, k)
    D = [t.double().requires_grad_() for t in (a["x"], a["wr"], a["bias"], *a["w"])]
    x, wr, bias, w0, w1, w2 = D
    weight = torch.softmax((x @ wr.t() + bias).gather(1, a["ids"]), 1)
    out = a["residual"].double()
    for j in range(k):
        e = a["ids"][:, j]
        g, u = (torch.einsum("th,tih->ti", x, m[e]) for m in (w0, w1))
        out = out + weight[:, j, None] * torch.einsum("ti,thi->th", g * torch.sigmoid(g) * u, w2[e])
    (out * a["dout"].double()).sum().backward()
    got = layer(**a, dtype=torch.bfloat16, how="act")
    want = dict(out=out.detach(), dx=x.grad + a["dx_in"].double(), dwr=wr.grad, db=bias.grad, dgate=w0.grad, dup=w1.grad,
                ddown=w2.grad)
    for n, v in got.items():
        # both in float64: 1e-10 of the largest
        assert float((v.v - want[n]).abs().max()) <= 1e-10 * float(want[n].abs().max()), n


MISTAKES = {"even weights": "out dgate dup ddown", "gate and up swapped": "out dx dgate dup ddown",
            "silu for its slope": "dx dgate", "no gradient through up": "dx", "no dx_in": "dx",
            "softmax without its mean": "dwr", "no gradient through the router": "dx"}


@pytest.mark.parametrize("how", ["act", "8bit"])
@pytest.mark.parametrize("mistake", MISTAKES)
def test_bounds_notice(mistake, how):
    """Some elements at least of each output that a mistake reaches are further off
    than their bounds, in bf16."""
    a = inputs(*CASES[0])
    want, wrong = (layer(**a, dtype=torch.bfloat16, how=how, mistake=m) for m in (None, mistake))
    for n in MISTAKES[mistake].split():
        assert bool(((want[n].v - wrong[n].v).abs() > want[n].e).any()), n
