"""MoELayerBuffers.layer_save and layer_backward (no GPU needed: the calls they
make are recorded instead of made)."""
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

T, H, E, I, K = 4, 256, 8, 128, 2


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in _abi.EXPORTS:
        if name in ("moe_workspace_size", "moe_train_workspace_size", "moe_status_str"):
            continue

        def record(*args, name=name, **kw):
            made.append((name, args))
            return 0

        monkeypatch.setattr(_abi, name, record, raising=False)
    return made


def t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def test_layer_save_then_backward(calls):
    buf = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    buf.layer_save(t(T, H), t(E, H), None, "experts", residual="res", kept="8bit")
    assert [n for n, _ in calls] == ["moe_route_permute", "moe_ffn_gate_up_save", "moe_ffn_down", "moe_combine"]
    assert buf.g.dtype == torch.int8 and buf.g_scale.shape == (T * K, I // 32)
    saved = buf.saved
    calls.clear()
    dx, dwr, db = t(T, H), t(E, H, dtype=torch.float32), t(E, dtype=torch.float32)
    buf.layer_backward("dout", "x", "wr", "experts", dx, dwr, db, "dexperts", dx_in="dx_in")
    assert [n for n, _ in calls] == ["moe_combine_backward", "moe_ffn_backward", "moe_dispatch_backward",
                                     "moe_router_backward"]
    ffn, disp, router = calls[1][1], calls[2][1], calls[3][1]
    # shape, dy, x, x_scale, saved, experts, perm, drows, dexperts
    assert ffn[1] is buf.dy and ffn[2] == "x" and ffn[3] is None and ffn[4] is saved
    assert ffn[7] is buf.drows and ffn[8] == "dexperts"
    # what reaches x through the experts is added to dx_in, and both to the router's
    assert disp[1] is buf.drows and disp[5] == "dx_in" and disp[6] is buf.dx_rows
    assert router[7] is buf.dx_rows and router[8] is dx and router[9] is dwr and router[10] is db


def test_a_checkpoint_of_x_is_read_back_once(calls):
    """The experts' gradient and the router's both take it."""
    buf = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    buf.layer_save(t(T, H), t(E, H), None, "experts")
    calls.clear()
    buf.layer_backward("dout", "codes", "wr", "experts", t(T, H), x_scale="scales")
    assert [n for n, _ in calls][0] == "moe_restore8" and sum(n == "moe_restore8" for n, _ in calls) == 1
    assert calls[0][1][3:6] == ("codes", "scales", buf.x_back)
    ffn = next(a for n, a in calls if n == "moe_ffn_backward")
    router = next(a for n, a in calls if n == "moe_router_backward")
    assert ffn[2] is buf.x_back and ffn[3] is None and router[4] is buf.x_back


def test_kept_memory_is_made_once(calls):
    buf = M.MoELayerBuffers(T, H, E, I, K, act="f32", device="cpu")
    buf.layer_save(t(T, H), t(E, H), None, "experts")
    g, ws = buf.g, buf.train_ws
    assert g.dtype == torch.float32 and buf.g_scale is None
    buf.layer_save(t(T, H), t(E, H), None, "experts")
    assert buf.g is g and buf.train_ws is ws
    buf.layer_save(t(T, H), t(E, H), None, "experts", kept="8bit")
    assert buf.g.dtype == torch.int8 and buf.train_ws is ws
    with pytest.raises(ValueError, match="kept"):
        buf.layer_save(t(T, H), t(E, H), None, "experts", kept="4bit")


def test_layer_save_refuses_a_buffer_that_has_to_check(calls):
    buf = M.MoELayerBuffers(T, H, E, I, K, device="cpu", check_finite=True)
    with pytest.raises(M.MoEError, match="MOE_E_FLAGS"):
        buf.layer_save(t(T, H), t(E, H), None, "experts")
    assert not calls
