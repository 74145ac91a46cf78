"""MoELayerBuffers.block and the options of its buffer (no GPU needed: the
calls it makes are recorded instead of made)."""
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
        if name in ("moe_workspace_size", "moe_status_str"):
            continue

        def record(*args, name=name, **kw):
            made.append((name, args))
            return 0

        monkeypatch.setattr(_abi, name, record, raising=False)
    return made


def block(buf, **kw):
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    pre, post = M.make_norm(T, H), M.make_norm(T, H)
    return buf.block(t(T, H), pre, t(H), t(E, H), None, "experts", post, t(H), n=t(T, H), **kw)


def test_block_refuses_a_buffer_that_has_to_check(calls):
    """Its steps do not check for NaN and infinity, and publish as they go."""
    with pytest.raises(M.MoEError, match="MOE_E_FLAGS") as e:
        block(M.MoELayerBuffers(T, H, E, I, K, device="cpu", check_finite=True))
    assert e.value.status == 10 and not calls


@pytest.mark.parametrize("fused", [False, True])
def test_block_runs_the_experts_its_buffer_asks_for(calls, fused):
    block(M.MoELayerBuffers(T, H, E, I, K, device="cpu", tiled=True, fused=fused))
    experts = ["moe_ffn_fused"] if fused else ["moe_ffn_gate_up", "moe_ffn_down"]
    assert [n for n, _ in calls] == ["moe_norm_in", "moe_route_permute", *experts, "moe_combine_norm"]


def test_block_keeps_the_branch(calls):
    """z, which the gradient of the norm after the block needs, reaches the
    combine; without it nothing is written there."""
    z = torch.zeros(T, H, dtype=torch.bfloat16)
    for kept in (z, None):
        calls.clear()
        block(M.MoELayerBuffers(T, H, E, I, K, device="cpu"), z=kept)
        name, args = calls[-1]
        # shape, norm, y, pair_row, topk_w, w, gate, residual, w_next, z, ...
        assert name == "moe_combine_norm" and args[9] is kept
