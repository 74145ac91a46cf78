"""Memory that MoELayerBuffers makes for training (no GPU needed: the calls are
replaced by ones that do nothing)."""
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

T, H, E, I, K = 4, 256, 8, 128, 2
SET = ("kept", "g", "u", "g_scale", "u_scale", "saved")


@pytest.fixture
def buf(monkeypatch):
    for name in _abi.EXPORTS:
        if name not in ("moe_workspace_size", "moe_train_workspace_size", "moe_status_str"):
            monkeypatch.setattr(_abi, name, lambda *args, **kw: 0, raising=False)
    return M.MoELayerBuffers(T, H, E, I, K, device="cpu")


def t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def save(buf, **kw):
    buf.layer_save(t(T, H), t(E, H), None, "experts", **kw)


def backward(buf, **kw):
    buf.layer_backward("dout", "x", "wr", "experts", t(T, H), **kw)


def now(buf):
    return [getattr(buf, n, None) for n in SET]


def test_each_form_keeps_its_memory(buf):
    """Work that is queued, or captured in a graph, may still write the other
    form's g and u."""
    save(buf)
    act = now(buf)
    save(buf, kept="8bit")
    q8 = now(buf)
    assert q8[0] == "8bit" and q8[1].dtype == torch.int8 and q8[1].data_ptr() != act[1].data_ptr()
    save(buf)
    assert all(a is b for a, b in zip(now(buf), act))
    save(buf, kept="8bit")
    assert all(a is b for a, b in zip(now(buf), q8))
    assert buf.saved.g == buf.g.data_ptr() and buf.saved.u_scale == buf.u_scale.data_ptr()


class OutOfMemory(RuntimeError):
    pass


@pytest.fixture
def fail_at(monkeypatch):
    """fail_at(n): the n-th allocation from now on fails, once."""
    left = []

    def count(fn):
        def empty(*args, **kw):
            if left:
                left[0] -= 1
                if left[0] == 0:
                    left.clear()
                    raise OutOfMemory
            return fn(*args, **kw)
        return empty

    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, count(getattr(torch, name)))

    def set_(n):
        left[:] = [n]
    return set_


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_a_failed_change_of_form_changes_nothing(buf, fail_at, n):
    save(buf)
    before = now(buf)
    fail_at(n)
    with pytest.raises(OutOfMemory):
        save(buf, kept="8bit")
    assert all(a is b for a, b in zip(now(buf), before))
    save(buf)
    assert all(a is b for a, b in zip(now(buf), before))
    save(buf, kept="8bit")
    assert all(v is not None for v in now(buf)) and buf.g_scale.shape == (T * K, I // 32)


@pytest.mark.parametrize("n", [1, 2, 3])
def test_a_failed_first_save_can_be_repeated(buf, fail_at, n):
    fail_at(n)
    with pytest.raises(OutOfMemory):
        save(buf)
    save(buf)
    assert buf.train_ws.numel() == buf.train_ws_bytes and buf.kept == "act"


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_a_failed_backward_can_be_repeated(buf, fail_at, n):
    save(buf)
    fail_at(n)
    with pytest.raises(OutOfMemory):
        backward(buf)
    backward(buf)
    assert buf.dy.shape == buf.drows.shape == (T * K, H) and buf.dw.shape == (T, K)
    assert buf.dx_rows.shape == (T, H)
