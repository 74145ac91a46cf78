"""layer_save and layer_backward as a whole, in bf16 and with g and u in 8 bits:
values against 64-bit definitions, of the layer from its inputs (tests/train_layer_ref.py)
and of each step from the tensors that the step before left (tests/train_ref.py)."""
import pytest
import torch

from tests import train_ref as R
from tests.test_gpu_train import DT, Layer
from tests.train_layer_ref import EW, layer

pytestmark = pytest.mark.gpu

FORMS = [("bf16", "act"), ("bf16", "8bit"), ("f32", "act"), ("f32", "8bit")]
SIZES = [(1, 128, 1, 32, 1), (50, 256, 12, 96, 3), (300, 128, 4, 64, 2), (7, 384, 64, 32, 5), (141, 640, 3, 160, 2)]


@pytest.mark.parametrize("act,kept", FORMS)
@pytest.mark.parametrize("T,H,E,I,k", SIZES)
def test_layer_gradients(T, H, E, I, k, act, kept):
    b = Layer(T, H, E, I, k, act, kept, seed=31)
    b.step()
    weight = torch.softmax((b.x.double() @ b.wr.double().t() + b.bias.double()).gather(1, b.buf.topk_ids.long()), 1)
    assert float((b.buf.topk_w.double() - weight).abs().max()) <= EW
    want = layer(b.x, b.wr, b.bias, b.w, b.buf.topk_ids, b.x, b.dout, b.dout, DT[act], kept)
    R.check({n: v for n, v in b.outputs().items() if n in want}, {n: (v.v, v.e) for n, v in want.items()},
            f"layer {T} {H} {E} {I} {k} {act} {kept}")


@pytest.mark.parametrize("act,kept", FORMS)
@pytest.mark.parametrize("T,H,E,I,k", SIZES)
def test_layer_steps(T, H, E, I, k, act, kept):
    dt = DT[act]
    b = Layer(T, H, E, I, k, act, kept, seed=32)
    b.step()
    buf, P, what = b.buf, T * k, f"{T} {H} {E} {I} {k} {act} {kept}"
    order, row = buf.sorted_pair.long(), buf.pair_row.long()
    token, ex = order // k, buf.topk_ids.reshape(-1).long()[order]
    want = R.gate_up(b.x, b.w[0], b.w[1], buf.offsets, buf.sorted_pair, k, dt)
    if kept == "act":
        g, u = buf.g, buf.u
        want.update({m: R._round(*want[m], dt) for m in ("g", "u")})
    else:
        g, u = R.values8(buf.g, buf.g_scale), R.values8(buf.u, buf.u_scale)
        for m, scale in (("g", buf.g_scale), ("u", buf.u_scale)):
            half = R.pow2(scale.long() - 127).repeat_interleave(32, 1) / 2
            want[m] = want[m][0], want[m][1] + half
    R.check(dict(g=g, u=u, h=buf.h), want, what)

    # y = W_down h, out = residual + sum w y
    h, wd, w = buf.h.double(), b.w[2].double(), buf.topk_w.double()
    y, ey = (torch.stack([f(m[e]) @ f(v) for e, v in zip(ex, h)]) if P else h.new_zeros(0, H)
             for f, m in ((lambda t: t, wd), (torch.abs, wd)))
    R.check({"y": buf.y}, {"y": R._round(y, 2 * (I + 2) * R.E * ey + I * R.TINY, dt)}, what)
    slots = lambda t: t.double()[row].reshape(T, k, -1)
    terms = w[:, :, None] * slots(buf.y)
    out, mag = b.x.double() + terms.sum(1), b.x.double().abs() + terms.abs().sum(1)
    R.check({"out": buf.out}, {"out": R._round(out, (k + 3) * R.E * mag, dt)}, what)

    # dy = w dout, dw = dout . y
    dout = b.dout.double()
    dy = (w.reshape(-1)[order])[:, None] * dout[token]
    R.check({"dy": buf.dy}, {"dy": R._round(dy, R.E * dy.abs(), dt)}, what)
    prod = dout[:, None, :] * slots(buf.y)
    R.check({"dw": buf.dw}, {"dw": (prod.sum(2), 2 * (H + 2) * R.E * prod.abs().sum(2) + H * R.TINY)}, what)

    want = R.backward(buf.dy, b.x, g, u, *b.w, buf.offsets, buf.sorted_pair, k, dt)
    R.check(dict(drows=buf.drows, dgate=b.dw[0], dup=b.dw[1], ddown=b.dw[2]), want, what)
    rows = slots(buf.drows)
    dx, mag = dout + rows.sum(1), dout.abs() + rows.abs().sum(1)
    R.check({"dx_rows": buf.dx_rows}, {"dx_rows": R._round(dx, (k + 3) * R.E * mag, dt)}, what)
    want = R.router(buf.topk_ids, buf.topk_w, buf.dw, b.x, b.wr, buf.dx_rows, dt)
    R.check(dict(dx=b.dx, dw_router=b.dwr, dbias=b.db), want, what)
