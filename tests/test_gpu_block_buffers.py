"""MoELayerBuffers.block on the GPU: the options of its buffer."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests.test_gpu_block import DEV, EPS, Gen, Out

pytestmark = pytest.mark.gpu


def block_inputs(T, H, E, I):
    """(x, router, tiled experts, both norm weights); the tensors behind the
    experts' addresses last."""
    g, bf = Gen(T, H, E, 61), torch.bfloat16
    ws = [g(E, *sh, std=0.05, dtype=bf) for sh in ((I, H), (I, H), (H, I))]
    dst = [torch.empty_like(w) for w in ws]
    M.moe_tile_experts(M.make_shape(T, H, E, I, 1), M.make_experts(*ws), M.make_experts(*dst))
    w1, w2 = g(H, std=0.1, mean=1.0, dtype=bf), g(H, std=0.1, mean=1.0, dtype=bf)
    return g(T, H, dtype=bf), g(E, H, std=0.05, dtype=bf), M.make_experts(*dst), w1, w2, dst


@pytest.mark.parametrize("T,H,E,I,k", [(1, 256, 16, 128, 2), (8, 512, 64, 128, 6), (130, 256, 16, 256, 3)])
def test_block_of_a_fused_buffer(T, H, E, I, k):
    """The bits of its steps with moe_ffn_fused between them."""
    x, wr, ex, w1, w2, _keep = block_inputs(T, H, E, I)
    pre, post = M.make_norm(T, H, eps=EPS), M.make_norm(T, H, eps=EPS)
    n, out, ref = (Out(T, H, dtype=torch.bfloat16) for _ in range(3))
    buf, other = (M.MoELayerBuffers(T, H, E, I, k, device=DEV, tiled=True, fused=True) for _ in range(2))
    buf.block(x, pre, w1, wr, None, ex, post, w2, residual=x, n=n.t, out=out.t)
    other.route_permute(n.t, wr, logits=False)
    other.ffn_fused(n.t, ex)
    other.combine_norm(post, w2, residual=x, out=ref.t)
    assert torch.equal(buf.y, other.y) and torch.equal(out.t, ref.t)
    assert out.t.isfinite().all() and n.ok() and out.ok()


@pytest.mark.parametrize("fused", [False, True])
def test_block_keeps_the_branch(fused):
    """z is the combine's own result, and the other outputs do not change."""
    T, H, E, I, k = 40, 256, 16, 128, 3
    x, wr, ex, w1, w2, _keep = block_inputs(T, H, E, I)
    pre, post = M.make_norm(T, H, eps=EPS), M.make_norm(T, H, eps=EPS)
    n, out, ref, z = (Out(T, H, dtype=torch.bfloat16) for _ in range(4))
    buf = M.MoELayerBuffers(T, H, E, I, k, device=DEV, tiled=True, fused=fused)
    buf.block(x, pre, w1, wr, None, ex, post, w2, residual=x, n=n.t, out=ref.t)
    buf.block(x, pre, w1, wr, None, ex, post, w2, residual=x, n=n.t, out=out.t, z=z.t)
    assert torch.equal(out.t, ref.t)
    buf.combine(out=ref.t)
    assert torch.equal(z.t, ref.t) and all(o.ok() for o in (n, out, ref, z))
