"""layer_save, layer_backward and the methods they call refuse before anything is
enqueued or made (no GPU needed: the calls are recorded instead of made)."""
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

T, H, E, I, K = 4, 256, 8, 128, 2
SIZES = ("moe_workspace_size", "moe_train_workspace_size", "moe_status_str")


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in _abi.EXPORTS:
        if name not in SIZES:
            monkeypatch.setattr(_abi, name, lambda *a, name=name, **kw: (made.append(name), 0)[1], raising=False)
    return made


def t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def methods(b):
    """Every way into the products."""
    return dict(layer_save=lambda: b.layer_save(t(T, H), t(E, H), None, "experts"),
                ffn_gate_up_save=lambda: b.ffn_gate_up_save("x", "experts"),
                layer_backward=lambda: b.layer_backward("dout", "x", "wr", "experts", "dx"),
                ffn_backward=lambda: b.ffn_backward("dy", "x", "experts", "drows"))


@pytest.mark.parametrize("kw,error", [
    (dict(tiled=True), "MOE_E_FLAGS"), (dict(tiled=True, fused=True), "MOE_E_FLAGS"),
    (dict(wfmt="int4_g32"), "MOE_E_FORMAT"), (dict(wfmt="int2_g32", tiled=True), "MOE_E_FORMAT")])
@pytest.mark.parametrize("name", ["layer_save", "ffn_gate_up_save", "layer_backward", "ffn_backward"])
def test_buffers_whose_products_are_refused(calls, kw, error, name):
    b = M.MoELayerBuffers(T, H, E, I, K, device="cpu", **kw)
    with pytest.raises(M.MoEError, match=error):
        methods(b)[name]()
    assert not calls and not hasattr(b, "train_ws") and not hasattr(b, "dy")


def test_sizes_past_the_products_limits(calls):
    """float32 token rows of 4 GiB, which the other steps take."""
    b = M.MoELayerBuffers(T, H, E, I, K, act="f32", device="cpu")
    b.shape = M.make_shape(131072, 8192, 4, 32, 1, "f32")
    for name in ("layer_save", "ffn_gate_up_save", "layer_backward", "ffn_backward"):
        with pytest.raises(M.MoEError, match="MOE_E_LIMIT"):
            methods(b)[name]()
    assert not calls and not hasattr(b, "train_ws")


@pytest.mark.parametrize("name", ["layer_backward", "ffn_backward"])
def test_a_gradient_before_its_products(calls, name):
    b = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    with pytest.raises(M.MoEError, match="before .*: MOE_E_NULL"):
        methods(b)[name]()
    assert not calls and not hasattr(b, "dy")
    b.layer_save(t(T, H), t(E, H), None, "experts")
    calls.clear()
    methods(b)[name]()
    assert calls


def test_a_form_that_is_not_known(calls):
    b = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    with pytest.raises(ValueError, match="kept"):
        b.layer_save(t(T, H), t(E, H), None, "experts", kept="4bit")
    assert not calls and not hasattr(b, "train_ws")


def test_the_routers_gradient_takes_any_weights(calls):
    """It reads no expert weights."""
    b = M.MoELayerBuffers(T, H, E, I, K, device="cpu", wfmt="int4_g32", tiled=True)
    b.router_backward("dw", "x", "wr", "dx")
    assert calls == ["moe_router_backward"] and b.train_ws_bytes > 0


def test_an_empty_batch(calls):
    b = M.MoELayerBuffers(0, H, E, I, K, device="cpu")
    b.layer_save(t(0, H), t(E, H), None, "experts")
    b.layer_backward("dout", "x", "wr", "experts", "dx")
    assert len(calls) == 8


def test_a_refused_save_keeps_the_last_one(calls, monkeypatch):
    b = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    b.layer_save(t(T, H), t(E, H), None, "experts")
    before = b.kept, b.g, b.u, b.g_scale, b.saved

    def refuse(*args, **kw):
        raise M.MoEError(5, "refused")

    for name in ("moe_ffn_gate_up_save", "moe_route_permute"):
        with monkeypatch.context() as m:
            m.setattr(_abi, name, refuse)
            with pytest.raises(M.MoEError, match="refused"):
                b.layer_save(t(T, H), t(E, H), None, "experts", kept="8bit")
        assert all(x is y for x, y in zip((b.kept, b.g, b.u, b.g_scale, b.saved), before))
