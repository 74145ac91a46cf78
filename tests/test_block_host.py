"""Refusals of the operators around the routed experts (no GPU needed): every
invalid call returns its status before anything is enqueued, and leaves its
outputs alone (host sentinel buffers stand in for device memory)."""
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi
from tests.test_abi_host import HostBuf

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE, FLAGS, MEMORY, VALUE = 1, 2, 3, 5, 6, 7, 10, 12, 13
TOKEN, FULL, SIG, NONORM = 1, 2, 4, 8
NAMES = ("a", "b", "c", "d", "e", "f", "g", "h", "i", "j", "k")


class Bufs(dict):
    def __init__(self):
        super().__init__({n: HostBuf(1 << 14) for n in NAMES})

    def at(self, name):
        return self[name].addr

    def untouched(self):
        return all(v.untouched() for v in self.values())


def norm(**kw):
    d = dict(T=4, H=96, act="bf16")
    d.update(kw)
    return M.make_norm(**d)


def shape(**kw):
    d = dict(T=4, H=128, E=8, I=64, top_k=2, act="bf16")
    d.update(kw)
    return M.make_shape(**d)


def call(fn, base, args, over):
    a = dict(args)
    a.update(over)
    return fn(*base, stream=0, check=False, **a)


CALLS = {
    "norm_in": (M.moe_norm_in, lambda: (norm(),), dict(x="a", w="b", n="c"), ("x", "w", "n"), ("n",)),
    "norm_in_backward": (M.moe_norm_in_backward, lambda: (norm(),),
                         dict(dn="a", x="b", w="c", dres="d", dx="e", dw="f", workspace="g",
                              workspace_bytes=1 << 20),
                         ("dn", "x", "w", "dx"), ("dx", "dw")),
    "norm_out": (M.moe_norm_out, lambda: (norm(flags=TOKEN),),
                 dict(z="a", w="b", gate="c", residual="d", w_next="e", out="f", n_next="g"),
                 ("z", "w", "gate", "out", "n_next", "w_next"), ("out", "n_next")),
    "norm_out_backward": (M.moe_norm_out_backward, lambda: (norm(flags=FULL | SIG),),
                          dict(dout="a", z="b", w="c", gate="d", dz="e", dgate="f", dw="g",
                               workspace="h", workspace_bytes=1 << 20),
                          ("dout", "z", "w", "gate", "dz"), ("dz", "dgate", "dw")),
    "combine_norm": (M.moe_combine_norm, lambda: (shape(), norm(H=128, flags=FULL)),
                     dict(y="a", pair_row="b", topk_w="c", w="d", gate="e", residual="f", w_next="g",
                          z="h", out="i", n_next="j"),
                     ("y", "pair_row", "topk_w", "w", "gate", "out", "w_next", "n_next"),
                     ("z", "out", "n_next")),
    "dispatch": (M.moe_dispatch, lambda: (shape(),), dict(x="a", pair_row="b", topk_w="c", rows="d"),
                 ("x", "pair_row", "rows"), ("rows",)),
    "dispatch_backward": (M.moe_dispatch_backward, lambda: (shape(),),
                          dict(drows="a", pair_row="b", topk_w="c", x="d", dx_in="e", dx="f", dw="g"),
                          ("drows", "pair_row", "topk_w", "x", "dx"), ("dx", "dw")),
    "combine_backward": (M.moe_combine_backward, lambda: (shape(),),
                         dict(dout="a", y="b", pair_row="c", topk_w="d", dy="e", dw="f"),
                         ("dout", "y", "pair_row", "topk_w", "dy"), ("dy", "dw")),
    "route_backward": (M.moe_route_backward, lambda: (shape(),),
                       dict(topk_ids="a", topk_w="b", dw="c", dlogits="d"),
                       ("topk_ids", "topk_w", "dw", "dlogits"), ("dlogits",)),
}


def addresses(b, args):
    return {k: (b.at(v) if isinstance(v, str) else v) for k, v in args.items()}


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    fn, base, args, required, outs = CALLS[name]
    b = Bufs()
    a = addresses(b, args)
    for arg in required:
        assert call(fn, base(), a, {arg: None}) == NULL, arg
    for arg, v in args.items():
        if isinstance(v, str):
            assert call(fn, base(), a, {arg: b.at(v) + 4}) == ALIGN, arg
    ins = [x for x, v in args.items() if isinstance(v, str) and x not in outs]
    for o in outs:
        for i in ins:
            assert call(fn, base(), a, {o: a[i]}) == ALIAS, (o, i)
        for o2 in outs:
            if o2 != o:
                assert call(fn, base(), a, {o: a[o2] + 16}) == ALIAS, (o, o2)
    assert b.untouched()


@pytest.mark.parametrize("name", ["norm_in_backward", "norm_out_backward"])
def test_workspace(name):
    fn, base, args, _, _ = CALLS[name]
    b = Bufs()
    a = addresses(b, args)
    need = M.moe_norm_workspace_size(base()[0])
    assert need >= 96 * 4
    assert call(fn, base(), a, dict(workspace_bytes=need - 1)) == WORKSPACE
    assert call(fn, base(), a, dict(workspace=None)) == WORKSPACE
    assert b.untouched()


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(H=0), SHAPE), (dict(H=65537), SHAPE),
    (dict(act=7), DTYPE), (dict(flags=16), FLAGS), (dict(flags=TOKEN | FULL), FLAGS),
    (dict(flags=SIG), FLAGS), (dict(eps=0.0), VALUE), (dict(eps=-1e-6), VALUE),
    (dict(eps=1e-40), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE),
    (dict(weight_offset=float("nan")), VALUE), (dict(residual_scale=float("inf")), VALUE),
    (dict(branch_scale=float("nan")), VALUE),
])
def test_descriptor(over, code):
    b = Bufs()
    n = norm(**over)
    assert M.moe_norm_workspace_size(n) == 0
    p = lambda *names: [b.at(x) for x in names]
    kw = dict(stream=0, check=False)
    assert M.moe_norm_in(n, *p("a", "b", "c"), **kw) == code
    assert M.moe_norm_in_backward(n, *p("a", "b", "c", "d", "e", "f", "g"), 1 << 20, **kw) == code
    assert M.moe_norm_out(n, *p("a", "b", "c", "d", "e", "f", "g"), **kw) == code
    assert M.moe_norm_out_backward(n, *p("a", "b", "c", "d", "e", "f", "g", "h"), 1 << 20, **kw) == code
    n.H = 128 if n.H == 96 else n.H
    if n.T == 4 and n.H == 128:
        assert M.moe_combine_norm(shape(), n, *p("a", "b", "c", "d", "e", "f", "g", "h", "i", "j"),
                                  **kw) == code
    assert b.untouched()


def test_null_descriptor():
    lib = M.load()
    assert lib.moe_norm_in(None, None, None, None, None) == NULL
    assert lib.moe_norm_in_backward(*(None,) * 8, 0, None) == NULL
    assert lib.moe_norm_out(*(None,) * 9) == NULL
    assert lib.moe_norm_out_backward(*(None,) * 9, 0, None) == NULL
    assert lib.moe_combine_norm(*(None,) * 13) == NULL
    assert lib.moe_dispatch(*(None,) * 6) == NULL
    assert lib.moe_dispatch_backward(*(None,) * 9) == NULL
    assert lib.moe_combine_backward(*(None,) * 8) == NULL
    assert lib.moe_route_backward(*(None,) * 6) == NULL
    assert lib.moe_norm_workspace_size(None) == 0


def test_flags_and_their_arguments():
    b = Bufs()
    p = lambda *names: [None if x is None else b.at(x) for x in names]
    kw = dict(stream=0, check=False)
    # norm_in takes no flags
    for f in (TOKEN, FULL, NONORM):
        assert M.moe_norm_in(norm(flags=f), *p("a", "b", "c"), **kw) == FLAGS
        assert M.moe_norm_in_backward(norm(flags=f), *p("a", "b", "c", "d", "e", "f", "g"), 1 << 20,
                                      **kw) == FLAGS
    # a gate or a weight without its flag, a flag without its gate
    assert M.moe_norm_out(norm(), *p("a", "b", "c", "d", "e", "f", "g"), **kw) == FLAGS
    assert M.moe_norm_out(norm(flags=NONORM), *p("a", "b", None, "d", "e", "f", "g"), **kw) == FLAGS
    assert M.moe_norm_out(norm(flags=FULL), *p("a", "b", None, "d", "e", "f", "g"), **kw) == NULL
    assert M.moe_norm_out(norm(), *p("a", None, None, "d", "e", "f", "g"), **kw) == NULL
    # dgate without a gate, dw without a norm
    assert M.moe_norm_out_backward(norm(), *p("a", "b", "c", None, "e", "f", "g", "h"), 1 << 20,
                                   **kw) == FLAGS
    assert M.moe_norm_out_backward(norm(flags=NONORM), *p("a", "b", None, None, "e", None, "g", "h"),
                                   1 << 20, **kw) == FLAGS
    # the norm's descriptor must describe the shape's rows
    args = p("a", "b", "c", "d", None, "f", "g", "h", "i", "j")
    assert M.moe_combine_norm(shape(), norm(H=256), *args, **kw) == SHAPE
    assert M.moe_combine_norm(shape(), norm(H=128, T=5), *args, **kw) == SHAPE
    assert M.moe_combine_norm(shape(), norm(H=128, act="f32"), *args, **kw) == DTYPE
    assert b.untouched()


def test_shape_domain():
    b = Bufs()
    kw = dict(stream=0, check=False)
    p = lambda *names: [b.at(x) for x in names]
    for over, code in ((dict(H=100), SHAPE), (dict(T=-1), SHAPE), (dict(top_k=9), SHAPE),
                       (dict(act=5), DTYPE), (dict(flags=64), FLAGS)):
        s = shape(**over)
        assert M.moe_dispatch(s, *p("a", "b", "c", "d"), **kw) == code
        assert M.moe_dispatch_backward(s, *p("a", "b", "c", "d", "e", "f", "g"), **kw) == code
        assert M.moe_combine_backward(s, *p("a", "b", "c", "d", "e", "f"), **kw) == code
        assert M.moe_route_backward(s, *p("a", "b", "c", "d"), **kw) == code
        assert M.moe_combine_norm(s, norm(H=128), *p("a", "b", "c", "d"), None,
                                  *p("f", "g", "h", "i", "j"), **kw) == code
    assert b.untouched()


def test_empty_batch():
    kw = dict(stream=0, check=False)
    n, s = norm(T=0), shape(T=0)
    assert M.moe_norm_workspace_size(n) == 0
    assert M.moe_norm_in(n, None, None, None, **kw) == 0
    assert M.moe_norm_in_backward(n, None, None, None, None, None, None, None, 0, **kw) == 0
    assert M.moe_norm_out(n, None, None, None, None, None, None, None, **kw) == 0
    assert M.moe_norm_out_backward(n, *(None,) * 8, 0, **kw) == 0
    assert M.moe_combine_norm(s, norm(T=0, H=128), *(None,) * 10, **kw) == 0
    assert M.moe_dispatch(s, None, None, None, None, **kw) == 0
    assert M.moe_dispatch_backward(s, *(None,) * 7, **kw) == 0
    assert M.moe_combine_backward(s, *(None,) * 6, **kw) == 0
    assert M.moe_route_backward(s, None, None, None, None, **kw) == 0
    assert M.moe_norm_in_backward(n, None, None, None, None, None, 4, None, 0, **kw) == ALIGN


def test_tensors_are_checked():
    """What a bare address cannot tell: type, size, layout, memory."""
    n = norm(T=4, H=96)
    kw = dict(stream=0, check=False)
    x = torch.zeros(4, 96, dtype=torch.bfloat16)
    w = torch.zeros(96, dtype=torch.bfloat16)
    out = torch.full((4, 96), 7, dtype=torch.bfloat16)
    assert M.moe_norm_in(n, x.float(), w, out, **kw) == DTYPE
    assert M.moe_norm_in(n, x.half(), w, out, **kw) == DTYPE
    assert M.moe_norm_in(n, x[:3], w, out, **kw) == SHAPE
    assert M.moe_norm_in(n, x, w[:95], out, **kw) == SHAPE
    assert M.moe_norm_in(n, torch.zeros(4, 192, dtype=torch.bfloat16)[:, ::2], w, out, **kw) == SHAPE
    assert M.moe_norm_in(n, torch.zeros(96, 4, dtype=torch.bfloat16).t(), w, out, **kw) == SHAPE
    assert M.moe_norm_in(n, x, w, out, **kw) == MEMORY            # host memory
    assert M.moe_norm_in_backward(n, x, x, w, None, out, torch.zeros(96, dtype=torch.float64), None, 0,
                                  **kw) == DTYPE
    gn = norm(T=4, H=96, flags=TOKEN)
    assert M.moe_norm_out(gn, x, w, torch.zeros(4, dtype=torch.bfloat16), None, None, out, None,
                          **kw) == DTYPE
    assert M.moe_norm_out(gn, x, w, torch.zeros(4, 96), None, None, out, None, **kw) == SHAPE
    s = shape()
    i64 = torch.zeros(8, dtype=torch.int64)
    xs, rows = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.bfloat16)
    assert M.moe_dispatch(s, xs, i64, None, rows, **kw) == DTYPE
    assert M.moe_dispatch(s, xs, i64.int(), torch.zeros(8), rows[:4], **kw) == SHAPE
    assert M.moe_route_backward(s, i64.int(), torch.zeros(8), torch.zeros(8), torch.zeros(4, 9),
                                **kw) == SHAPE
    ws = torch.zeros(16, dtype=torch.uint8)
    assert M.moe_norm_in_backward(n, 16, 32, 48, None, 64, 80, ws, 1 << 20, **kw) == WORKSPACE
    assert (out == 7).all()
    with pytest.raises(M.MoEError, match="moe_norm_in: MOE_E_SHAPE"):
        M.moe_norm_in(n, x[:3], w, out, stream=0)


def test_binding_arguments():
    """Arguments of the wrong kind raise; sizes whose product passes 64 bits
    match no tensor; without a stream the checks still answer."""
    x, w = torch.zeros(4, 96, dtype=torch.bfloat16), torch.zeros(96, dtype=torch.bfloat16)
    for bad in (1.5, "x", [x]):
        with pytest.raises(TypeError):
            M.moe_norm_in(norm(), bad, w, x, stream=0)
    for bad in (None, shape(), 16):
        with pytest.raises(TypeError):
            M.moe_norm_in(bad, x, w, x, stream=0)
        with pytest.raises(TypeError):
            M.moe_norm_in_backward(norm(), x, x, w, None, x, None, None, x, stream=0)
    # 2^22 * 2^22 * 2^20 elements: 0 modulo 2^64
    s = shape(T=1 << 22, top_k=1 << 22, H=1 << 20)
    empty = torch.zeros(0, dtype=torch.bfloat16)
    assert M.moe_combine_backward(s, None, empty, None, None, None, None, stream=0,
                                  check=False) == SHAPE
    assert M.moe_norm_in(norm(), x.float(), w, x, check=False) == DTYPE
    assert M.moe_norm_in(norm(), x, w, x.clone(), check=False) == MEMORY
