"""The stream that memory belongs to which a call of MoELayerBuffers makes: the
one that the call uses (no GPU needed for the first half: the calls are replaced by
ones that do nothing, and streams are recorded)."""
import contextlib
import os

import pytest
import torch

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")

T, H, E, I, K = 4, 256, 8, 128, 2


@pytest.fixture
def made(monkeypatch):
    """[stream] of every allocation, None for the current one."""
    for name in _abi.EXPORTS:
        if name not in ("moe_workspace_size", "moe_train_workspace_size", "moe_status_str",
                        "moe_route_locality_blocks"):
            monkeypatch.setattr(_abi, name, lambda *args, **kw: 0, raising=False)
    streams, on = [], [None]

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("handle", handle))
    for name in ("empty", "empty_like"):
        fn = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, fn=fn, **kw: (streams.append(on[-1]), fn(*a, **kw))[1])
    return streams


def t(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


@pytest.mark.parametrize("given,owner", [("a stream", "a stream"), (1234, ("handle", 1234)), (None, None)])
def test_memory_belongs_to_the_calls_stream(made, given, owner):
    buf = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
    assert set(made) == {None}                                  # the buffer's own: the current stream
    made.clear()
    buf.layer_save(t(T, H), t(E, H), None, "experts", stream=given)
    assert made == [owner] * 3                                  # workspace, g, u
    buf.layer_save(t(T, H), t(E, H), None, "experts", kept="8bit", stream=given)
    assert made == [owner] * 7                                  # and the other form's, with scales
    buf.layer_backward("dout", "codes", "wr", "experts", t(T, H), x_scale="scales", stream=given)
    assert made == [owner] * 12                                 # dy, drows, dw, dx_rows, x_back
    buf.route_locality(stream=given)
    assert made == [owner] * 14
    buf.layer_save(t(T, H), t(E, H), None, "experts", stream="another")
    buf.layer_backward("dout", "codes", "wr", "experts", t(T, H), x_scale="scales", stream="another")
    buf.route_locality(stream="another")
    assert len(made) == 14                                      # made once


def test_single_calls_too(made):
    for call in (lambda b: b.ffn_gate_up_save("x", "experts", stream="s"),
                 lambda b: b.router_backward("dw", "x", "wr", "dx", stream="s")):
        buf = M.MoELayerBuffers(T, H, E, I, K, device="cpu")
        made.clear()
        call(buf)
        assert made and set(made) == {"s"}


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_memory_comes_from_the_streams_pool(as_handle):
    """What a step makes lies in segments of its stream, also where the current
    stream has free memory of the same sizes."""
    dev = torch.device("cuda")
    shape = (600, 512, 8, 256, 2)

    def run(stream):
        T, H, E, I, K = shape
        buf = M.MoELayerBuffers(*shape, device=dev)
        g = torch.Generator(device=dev).manual_seed(1)
        r = lambda *s: (torch.randn(*s, generator=g, device=dev) * 0.1).bfloat16()
        x, wr, w = r(T, H), r(E, H), [r(E, I, H), r(E, I, H), r(E, H, I)]
        dx, codes, scales = torch.empty_like(x), *(torch.empty(T, n, dtype=d, device=dev)
                                                   for n, d in ((H, torch.int8), (H // 32, torch.uint8)))
        torch.cuda.synchronize()
        M.moe_save8("bf16", T, H, x, codes, scales, stream=stream)
        for kept in ("act", "8bit"):
            buf.layer_save(x, wr, None, M.make_experts(*w), kept=kept, stream=stream)
        buf.layer_backward(x, codes, wr, M.make_experts(*w), dx, x_scale=scales, stream=stream)
        buf.route_locality(stream=stream)
        torch.cuda.synchronize()
        return buf

    def owners(buf):
        mem = [buf.train_ws, buf.dy, buf.drows, buf.dw, buf.dx_rows, buf.x_back, buf.overlap_prev, buf.block_unique]
        mem += [v for s in buf._kept_sets.values() for v in s[:4] if v is not None]
        segments = torch.cuda.memory_snapshot()
        owner = lambda p: next(s["stream"] for s in segments if s["address"] <= p < s["address"] + s["total_size"])
        return {owner(v.data_ptr()) for v in mem}

    current = torch.cuda.current_stream().cuda_stream
    assert owners(run(None)) == {current}
    # all of it is free now, in the current stream's pool
    side = torch.cuda.Stream()
    assert owners(run(side.cuda_stream if as_handle else side)) == {side.cuda_stream}


@pytest.mark.gpu
def test_the_default_streams_handle():
    """A handle of 0 is the default stream."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(2)
    r = lambda *s: (torch.randn(*s, generator=g, device=dev) * 0.1).bfloat16()
    x, wr, w = r(T, H), r(E, H), [r(E, I, H), r(E, I, H), r(E, H, I)]
    got = []
    for stream in (None, 0, torch.cuda.default_stream()):
        buf, dx = M.MoELayerBuffers(T, H, E, I, K, device=dev), torch.empty_like(x)
        buf.layer_save(x, wr, None, M.make_experts(*w), stream=stream)
        buf.layer_backward(x, x, wr, M.make_experts(*w), dx, stream=stream)
        torch.cuda.synchronize()
        got.append((buf.out, dx))
    assert all(torch.equal(a, b) for other in got[1:] for a, b in zip(got[0], other))


@pytest.mark.gpu
def test_memory_made_while_a_graph_is_captured():
    """The first step of a buffer may be a captured one: replays and eager steps between
    them agree, with memory freed and taken again in between."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(4)
    r = lambda *s: (torch.randn(*s, generator=g, device=dev) * 0.1).bfloat16()
    T, H, E, I, K = 70, 256, 6, 96, 2
    x, wr, w = r(T, H), r(E, H), [r(E, I, H), r(E, I, H), r(E, H, I)]
    dx, dw = torch.empty_like(x), [torch.empty_like(t) for t in w]
    ex, dex = M.make_experts(*w), M.make_experts(*dw)

    def step(buf, kept):
        buf.layer_save(x, wr, None, ex, kept=kept)
        buf.layer_backward(x, x, wr, ex, dx, dexperts=dex)

    want = {}
    for kept in ("act", "8bit"):
        other = M.MoELayerBuffers(T, H, E, I, K, device=dev)
        step(other, kept)
        torch.cuda.synchronize()
        want[kept] = [t.clone() for t in (other.out, dx, *dw)]
    buf, graphs = M.MoELayerBuffers(T, H, E, I, K, device=dev), {}
    for kept in ("act", "8bit"):
        graphs[kept] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[kept]):
            step(buf, kept)
    for _ in range(3):
        for kept in ("8bit", "act"):
            for run in (graphs[kept].replay, lambda: step(buf, kept), graphs[kept].replay):
                for t in (buf.out, dx, *dw):
                    t.fill_(7)
                torch.full((1 << 20,), 3.0, device=dev)            # taken and given back
                run()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip((buf.out, dx, *dw), want[kept])), kept
