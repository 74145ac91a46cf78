"""Refusals of the training calls (no GPU needed): every invalid call returns
its status before anything is enqueued, and leaves its outputs alone (host
sentinel buffers stand in for device memory)."""
import ctypes
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi
from tests.test_abi_host import HostBuf

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

NULL, SHAPE, DTYPE, FORMAT, ALIGN, ALIAS, WORKSPACE, LIMIT, FLAGS, MEMORY = 1, 2, 3, 4, 5, 6, 7, 8, 10, 12
KW = dict(stream=0, check=False)


def shape(**kw):
    d = dict(T=4, H=128, E=8, I=64, top_k=2, act="bf16")
    d.update(kw)
    return M.make_shape(**d)


STRUCT = {"experts": (M.moe_experts, ("gate", "up", "down")), "dexperts": (M.moe_experts, ("gate", "up", "down")),
          "perm": (M.moe_perm, ("offsets", "sorted_pair")),
          "saved": (M.moe_saved, ("g", "u", "g_scale", "u_scale"))}
CALLS = {
    "save8": (M.moe_save8, ("v", "codes", "scales"), ("v", "codes", "scales"), ("codes", "scales")),
    "restore8": (M.moe_restore8, ("codes", "scales", "v"), ("v", "codes", "scales"), ("v",)),
    "gate_up_save": (M.moe_ffn_gate_up_save, ("x", "experts", "perm", "saved", "h", "workspace"),
                     ("x", "experts.gate", "experts.up", "perm.offsets", "perm.sorted_pair", "saved.g", "saved.u",
                      "saved.g_scale", "saved.u_scale", "h"),
                     ("h", "saved.g", "saved.u", "saved.g_scale", "saved.u_scale", "workspace")),
    "ffn_backward": (M.moe_ffn_backward,
                     ("dy", "x", "x_scale", "saved", "experts", "perm", "drows", "dexperts", "workspace"),
                     ("dy", "x", "experts.gate", "experts.up", "experts.down", "perm.offsets", "perm.sorted_pair",
                      "saved.g", "saved.u", "saved.g_scale", "saved.u_scale", "dexperts.gate", "dexperts.up",
                      "dexperts.down"),
                     ("drows", "dexperts.gate", "dexperts.up", "dexperts.down", "workspace")),
    "router_backward": (M.moe_router_backward,
                        ("topk_ids", "topk_w", "dw", "x", "w_router", "perm", "dx_in", "dx", "dw_router", "dbias",
                         "workspace"),
                        ("topk_ids", "topk_w", "dw", "x", "w_router", "perm.offsets", "perm.sorted_pair"),
                        ("dx", "dw_router", "dbias", "workspace")),
}


class Set:
    """Sentinel buffers for one call, by path (name, or struct.field)."""

    def __init__(self, name):
        self.fn, self.names, self.required, self.outs = CALLS[name]
        self.bufs = {}
        for n in self.names:
            for p in ([f"{n}.{f}" for f in STRUCT[n][1]] if n in STRUCT else [n]):
                self.bufs[p] = HostBuf(1 << 17)
        self.addr = {p: b.addr for p, b in self.bufs.items()}

    def __call__(self, s, over=None, drop=(), ws_bytes=1 << 17):
        addr = dict(self.addr, **(over or {}))
        args = []
        for n in self.names:
            if n in drop:
                args.append(None)
            elif n in STRUCT:
                cls, fields = STRUCT[n]
                args.append(cls(**{f: addr[f"{n}.{f}"] for f in fields}))
            else:
                args.append(addr[n])
        head = (s,) if isinstance(s, M.moe_shape) else tuple(s)
        tail = (ws_bytes,) if "workspace" in self.names else ()
        return self.fn(*head, *args, *tail, **KW)

    def untouched(self):
        return all(b.untouched() for b in self.bufs.values())


def base(name):
    return ("bf16", 8, 64) if name in ("save8", "restore8") else shape()


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    c = Set(name)
    for p in c.required:
        assert c(base(name), {p: None}) == NULL, p
    for p in c.addr:
        if name == "gate_up_save" and p == "experts.down":
            continue                                   # not read
        want = WORKSPACE if p == "workspace" else ALIGN
        if p == "workspace":
            assert c(base(name), {p: None}) == WORKSPACE
            want = ALIGN
        assert c(base(name), {p: c.addr[p] + 4}) == want, p
    ins = [p for p in c.addr if p not in c.outs and not (name == "gate_up_save" and p == "experts.down")]
    for o in c.outs:
        for p in ins:
            assert c(base(name), {o: c.addr[p]}) == ALIAS, (o, p)
        for o2 in c.outs:
            if o2 != o:
                assert c(base(name), {o: c.addr[o2]}) == ALIAS, (o, o2)
    assert c.untouched()


@pytest.mark.parametrize("name", ["gate_up_save", "ffn_backward", "router_backward"])
def test_structs_and_workspace(name):
    c = Set(name)
    for n in c.names:
        if n in STRUCT and n != "dexperts":
            assert c(shape(), drop=(n,)) == NULL, n
    need = M.moe_train_workspace_size(shape())
    assert need > 0
    assert c(shape(), ws_bytes=need - 1) == WORKSPACE
    assert c.untouched()


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), SHAPE), (dict(T=131073), SHAPE), (dict(H=96), SHAPE), (dict(I=48), SHAPE), (dict(E=1025), SHAPE),
    (dict(top_k=9), SHAPE), (dict(act=5), DTYPE), (dict(wfmt=9), FORMAT), (dict(flags=1 << 20), FLAGS)])
def test_descriptor(over, code):
    s = shape(**over)
    assert M.moe_train_workspace_size(s) == 0
    for name in ("gate_up_save", "ffn_backward", "router_backward"):
        c = Set(name)
        assert c(s) == code, name
        assert c.untouched()


@pytest.mark.parametrize("name", ["gate_up_save", "ffn_backward"])
def test_weight_formats(name):
    """The products take dense row-major weights; the router's gradient any."""
    c = Set(name)
    assert c(shape(wfmt="int4_g32")) == FORMAT
    assert c(shape(I=128, flags=M.MOE_F_TILED_WEIGHTS)) == FLAGS
    for p in ("experts", "dexperts"):
        if p in c.names:
            ex = M.moe_experts(*(c.addr[f"{p}.{f}"] for f in ("gate", "up", "down")), None, c.addr[c.names[0]], None)
            args = [ex if n == p else STRUCT[n][0](**{f: c.addr[f"{n}.{f}"] for f in STRUCT[n][1]}) if n in STRUCT
                    else c.addr[n] for n in c.names]
            assert c.fn(shape(), *args, 1 << 17, **KW) == FORMAT, p
    assert c.untouched()


def test_limits():
    """Offsets of float32 token rows are 32 bits; the tile counts stay under 2^23."""
    over = dict(T=131072, H=8192, I=32, E=4, top_k=1, act="f32")
    for name in ("gate_up_save", "ffn_backward"):
        c = Set(name)
        assert c(shape(**over)) == LIMIT
        assert c(shape(T=1, H=65536, I=65536, E=1024, top_k=1)) == LIMIT
        # bf16 rows of the same matrix fit: the next check answers
        assert c(shape(**dict(over, act="bf16"))) == WORKSPACE
        assert c.untouched()


def test_scales_come_in_pairs():
    for name in ("gate_up_save", "ffn_backward"):
        c = Set(name)
        assert c(shape(), {"saved.g_scale": None}) == NULL
        assert c(shape(), {"saved.u_scale": None}) == NULL


def test_what_may_be_left_out():
    c = Set("ffn_backward")
    assert c(shape(), {"drows": None}, drop=("dexperts",)) == NULL
    assert c(shape(), {"drows": None, "x": None}) == NULL            # dexperts needs x
    # without dexperts x is not needed: the next check answers
    assert c(shape(), {"x": None, "x_scale": None}, drop=("dexperts",), ws_bytes=0) == WORKSPACE
    c = Set("router_backward")
    assert c(shape(), {"dx": None, "dw_router": None, "dbias": None}) == NULL
    assert c(shape(), {"w_router": None}) == NULL
    assert c(shape(), {"w_router": None, "dx": None}, ws_bytes=0) == WORKSPACE
    assert c(shape(), {"x": None, "dw_router": None}, ws_bytes=0) == WORKSPACE
    assert c(shape(), {"dw_router": None, "dbias": None}, drop=("perm",), ws_bytes=0) == WORKSPACE
    assert c(shape(), {"dw_router": None}, drop=("perm",)) == NULL   # dbias needs perm
    assert c.untouched()


@pytest.mark.parametrize("name", ["save8", "restore8"])
def test_checkpoint_sizes(name):
    c = Set(name)
    assert c((7, 8, 64)) == DTYPE
    for rows, cols in ((-1, 64), (8, 0), (8, 33), (8, -32), (8, 16)):
        assert c(("bf16", rows, cols)) == SHAPE, (rows, cols)
    assert c(("f32", 1 << 36, 32)) == LIMIT
    assert c(("f32", (1 << 62), 32)) == LIMIT
    assert c(("bf16", 0, 64), {p: None for p in c.addr}) == 0       # nothing to do
    assert c.untouched()


def test_empty_batch():
    assert M.moe_train_workspace_size(shape(T=0)) == 0
    c = Set("gate_up_save")
    assert c(shape(T=0), {p: None for p in c.addr}) == 0
    c = Set("ffn_backward")
    assert c(shape(T=0), {p: None for p in c.addr if not p.startswith("drows")}, drop=("dexperts",)) == 0
    assert c(shape(T=0), {"dexperts.gate": None}) == NULL
    assert c(shape(T=0), {"dexperts.gate": c.addr["dexperts.up"]}) == ALIAS
    c = Set("router_backward")
    assert c(shape(T=0), {"dw_router": None, "dbias": None}) == 0
    assert c(shape(T=0), {"dw_router": c.addr["dbias"]}) == ALIAS
    assert c.untouched()


def test_workspace_size_covers_its_regions():
    s = shape(T=512, H=2560, E=512, I=640, top_k=10)
    P = 512 * 10
    assert M.moe_train_workspace_size(s) >= 3 * P * 640 * 2 + 512 * 2560 * 2
    # any valid shape has one: the router's gradient takes every weight format
    assert M.moe_train_workspace_size(shape(wfmt="int2_g32")) > 0
    assert M.moe_train_workspace_size(shape(I=128, flags=M.MOE_F_TILED_WEIGHTS)) > 0


def test_tensors_are_checked():
    """Type, size, layout and memory of tensors, as for the other compiled calls."""
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    ok = dict(v=t(8, 64), codes=t(8, 64, dtype=torch.int8), scales=t(8, 2, dtype=torch.uint8))
    call = lambda **kw: M.moe_save8("bf16", 8, 64, **dict(ok, **kw), **KW)
    assert call() == MEMORY                                          # host memory
    assert call(v=t(8, 64, dtype=torch.float32)) == DTYPE
    assert call(codes=t(8, 64, dtype=torch.uint8)) == DTYPE
    assert call(scales=t(8, 2, dtype=torch.int8)) == DTYPE
    assert call(v=t(64, 8).t()) == SHAPE
    assert call(scales=t(8, 3, dtype=torch.uint8)) == SHAPE
    s = shape()
    P, w = 8, torch.zeros(1 << 20, dtype=torch.uint8)
    ex, pm = M.make_experts(1 << 20, 1 << 21, 1 << 22), M.moe_perm(offsets=1 << 23, sorted_pair=1 << 24)
    sv = M.make_saved(1 << 25, 1 << 26)
    back = lambda dy=t(P, 128), x=t(4, 128), xs=None, drows=t(P, 128): M.moe_ffn_backward(
        s, dy, x, xs, sv, ex, pm, drows, None, w, 1 << 20, **KW)
    assert back() == MEMORY
    assert back(x=t(4, 128, dtype=torch.int8)) == DTYPE              # codes need their scales
    assert back(xs=t(4, 4, dtype=torch.uint8)) == DTYPE              # and scales codes
    assert back(x=t(4, 128, dtype=torch.int8), xs=t(4, 4, dtype=torch.uint8)) == MEMORY
    assert back(drows=t(P, 64)) == SHAPE
    assert back(dy=t(P - 1, 128)) == SHAPE
    assert M.moe_ffn_backward(s, t(P, 128), t(4, 128), None, sv, ex, pm, t(P, 128), None, w, 1 << 21,
                              **KW) == WORKSPACE
    with pytest.raises(TypeError):
        M.moe_ffn_backward(s, t(P, 128), t(4, 128), None, ex, ex, pm, t(P, 128), None, w, 1 << 20, **KW)
    with pytest.raises(M.MoEError, match="MOE_E_MEMORY"):
        M.moe_save8("bf16", 8, 64, **ok, stream=0)


def test_null_descriptor():
    lib = M.load()
    assert lib.moe_train_workspace_size(None) == 0
    assert lib.moe_ffn_gate_up_save(*(None,) * 7, 0, None) == NULL
    assert lib.moe_ffn_backward(*(None,) * 10, 0, None) == NULL
    assert lib.moe_router_backward(*(None,) * 12, 0, None) == NULL
    assert lib.moe_save8(1, 8, 64, None, None, None, None) == NULL
    assert ctypes.sizeof(M.moe_saved) == 32
