"""The memory that the training calls write through a descriptor (moe_saved, the
gradients' moe_experts) is checked like the tensors beside it: type, size, layout,
device (no GPU needed but for the last test: every call is refused)."""
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

DTYPE, SHAPE, MEMORY, FORMAT = 3, 2, 12, 4
T, H, E, I, K = 4, 128, 8, 64, 2
P = T * K
BF, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8
A = 1 << 20                       # an address: such arguments are taken as they are


def t(*s, dtype=BF):
    return torch.zeros(s, dtype=dtype)


def save(saved, act="bf16", **kw):
    return M.moe_ffn_gate_up_save(M.make_shape(T, H, E, I, K, act), A, M.make_experts(A, A, None),
                                  M.moe_perm(offsets=A, sorted_pair=A), saved, A, A, 1 << 30, stream=0, check=False)


def backward(saved=None, dexperts=None, act="bf16"):
    return M.moe_ffn_backward(M.make_shape(T, H, E, I, K, act), A, A, None, saved or M.make_saved(A, A),
                              M.make_experts(A, A, A), M.moe_perm(offsets=A, sorted_pair=A), A, dexperts, A, 1 << 30,
                              stream=0, check=False)


@pytest.mark.parametrize("call", [save, backward])
def test_saved(call):
    g, q, s = lambda: t(P, I), lambda: t(P, I, dtype=I8), lambda: t(P, I // 32, dtype=U8)
    # right, but for being host memory
    assert call(M.make_saved(g(), g())) == MEMORY
    assert call(M.make_saved(q(), q(), s(), s())) == MEMORY
    assert call(M.make_saved(t(P, I, dtype=F32), t(P, I, dtype=F32)), act="f32") == MEMORY
    # codes without their scales would be written in the activation type, past their end
    assert call(M.make_saved(q(), q())) == DTYPE
    assert call(M.make_saved(g(), q())) == DTYPE
    assert call(M.make_saved(g(), g(), s(), s())) == DTYPE
    assert call(M.make_saved(q(), q(), q(), s())) == DTYPE
    assert call(M.make_saved(q(), q(), s(), t(P, I // 32))) == DTYPE
    assert call(M.make_saved(g(), g()), act="f32") == DTYPE
    # too small, or not dense
    assert call(M.make_saved(t(P - 1, I), g())) == SHAPE
    assert call(M.make_saved(g(), t(P, I - 1))) == SHAPE
    assert call(M.make_saved(q(), q(), s(), t(P, 1, dtype=U8))) == SHAPE
    assert call(M.make_saved(g(), t(I, P).t())) == SHAPE
    assert call(M.make_saved(t(P, 2 * I)[:, :I], g())) == SHAPE
    # more memory than needed is fine, and so is a view that is gone
    assert call(M.make_saved(t(P + 9, I), g())) == MEMORY
    assert call(M.make_saved(t(3, P, I)[1], g())) == MEMORY


def test_the_weights_gradients():
    ok = lambda dtype=BF: [t(E, I, H, dtype=dtype), t(E, I, H, dtype=dtype), t(E, H, I, dtype=dtype)]
    assert backward(dexperts=M.make_experts(*ok())) == MEMORY
    assert backward(dexperts=M.make_experts(*ok(F32)), act="f32") == MEMORY
    assert backward(dexperts=M.make_experts(*ok(F32))) == DTYPE
    assert backward(dexperts=M.make_experts(*ok()), act="f32") == DTYPE
    for i in range(3):
        for wrong, code in ((t(E, I, H - 1), SHAPE), (t(E, I, H, dtype=torch.int16), DTYPE),
                            (t(H, E, I).permute(1, 2, 0), SHAPE), (t(E, I, 2 * H)[:, :, :H], SHAPE)):
            w = ok()
            w[i] = wrong
            assert backward(dexperts=M.make_experts(*w)) == code, (i, wrong.shape)


def test_a_field_that_was_set_by_hand_is_an_address():
    """Addresses carry no type, as everywhere: the next check answers."""
    s = M.make_saved(t(P, I, dtype=I8), t(P, I, dtype=I8))
    s.g = s.u = A
    d = M.make_experts(A, A, A, None, A)
    assert backward(s, d) == FORMAT
    assert backward(M.moe_saved(A, A), d) == FORMAT


def test_weights_that_are_read_are_taken_as_before():
    """make_experts of weights serves every call; what a call only reads is not
    looked at."""
    ex = M.make_experts(t(2, dtype=I8), t(2, dtype=U8), None)
    st = M.moe_ffn_gate_up_save(M.make_shape(T, H, E, I, K), A, ex, M.moe_perm(offsets=A, sorted_pair=A),
                                M.make_saved(A, A), A, None, 0, stream=0, check=False)
    assert st == 7                                             # no workspace


def test_descriptors_hold_no_memory():
    import gc
    import weakref
    w = [t(E, I, H) for _ in range(3)]
    d, alive = M.make_experts(*w), [weakref.ref(x) for x in w]
    del w
    gc.collect()
    assert d.gate and not any(a() is not None for a in alive)


@pytest.mark.gpu
def test_on_the_gpu():
    dev = torch.device("cuda")
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=dev)
    shape = M.make_shape(T, H, E, I, K)
    offsets = torch.arange(E + 1, dtype=torch.int32, device=dev)
    pair = torch.arange(P, dtype=torch.int32, device=dev)
    perm = M.make_perm(None, offsets, pair, None, None, None)
    ws = z(M.moe_train_workspace_size(shape), dtype=U8)
    w = [z(E, I, H), z(E, I, H), z(E, H, I)]               # descriptors hold no memory
    ex = M.make_experts(*w)
    x, h, dy, drows = z(T, H), z(P, I), z(P, H), z(P, H)

    def calls(saved, dex):
        return (M.moe_ffn_gate_up_save(shape, x, ex, perm, saved, h, ws, ws.numel(), check=False),
                M.moe_ffn_backward(shape, dy, x, None, saved, ex, perm, drows, dex, ws, ws.numel(), check=False))

    keep = [z(P, I, dtype=I8), z(P, I, dtype=I8), z(P, I // 32, dtype=U8), z(P, I // 32, dtype=U8)]
    dw = [z(E, I, H), z(E, I, H), z(E, H, I)]
    assert calls(M.make_saved(*keep), M.make_experts(*dw)) == (0, 0)
    assert calls(M.make_saved(*keep[:2]), M.make_experts(*dw)) == (DTYPE, DTYPE)
    assert calls(M.make_saved(z(P, I), z(P, I).cpu()), M.make_experts(*dw)) == (MEMORY, MEMORY)
    assert calls(M.make_saved(*keep), M.make_experts(dw[0], dw[1], dw[2].mT)) == (0, SHAPE)
    assert calls(M.make_saved(*keep), M.make_experts(dw[0].cpu(), dw[1], dw[2])) == (0, MEMORY)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_pinned_host_memory():
    """g, u and a gradient in pinned host memory, which the GPU writes: the values of
    the same call with memory of the GPU."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device=dev).bfloat16()
    shape = M.make_shape(T, H, E, I, K)
    offsets = torch.arange(E + 1, dtype=torch.int32, device=dev)
    pair = torch.arange(P, dtype=torch.int32, device=dev)
    perm = M.make_perm(None, offsets, pair, None, None, None)
    ws = torch.empty(M.moe_train_workspace_size(shape), dtype=U8, device=dev)
    w, x, dy = [r(E, I, H), r(E, I, H), r(E, H, I)], r(T, H), r(P, H)
    h, drows = torch.empty(P, I, dtype=BF, device=dev), torch.empty(P, H, dtype=BF, device=dev)
    got = []
    for where in (dict(device=dev), dict(pin_memory=True)):
        keep = [torch.empty(P, I, dtype=BF, **where) for _ in range(2)]
        dw = [torch.empty(s, dtype=BF, **where) for s in ((E, I, H), (E, I, H), (E, H, I))]
        saved = M.make_saved(*keep)
        M.moe_ffn_gate_up_save(shape, x, M.make_experts(*w), perm, saved, h, ws, ws.numel())
        M.moe_ffn_backward(shape, dy, x, None, saved, M.make_experts(*w), perm, drows, M.make_experts(*dw), ws,
                           ws.numel())
        torch.cuda.synchronize()
        got.append([t.cpu() for t in (*keep, *dw, drows)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
