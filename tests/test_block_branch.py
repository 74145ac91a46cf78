"""moe_norm_out_backward: when z may be NULL, and what is still refused (no
GPU needed)."""
import os

import pytest

import sparse_moe_routed_amd as M
from sparse_moe_routed_amd import _abi
from tests.test_block_host import ALIAS, ALIGN, FULL, NONORM, NULL, SIG, TOKEN, Bufs, norm

pytestmark = pytest.mark.skipif(not os.path.exists(_abi.LIB_PATH),
                                reason="libmoe.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("flags", [0, TOKEN, FULL, FULL | SIG])
def test_branch_that_is_read_is_required(flags):
    b = Bufs()
    kw = dict(stream=0, check=False)
    gate = b.at("d") if flags else None
    # a norm reads z, with or without gradients beside dz
    n = norm(flags=flags)
    assert M.moe_norm_out_backward(n, b.at("a"), None, b.at("c"), gate, b.at("e"), None, None, None, 0,
                                   **kw) == NULL
    n = norm(flags=flags | NONORM)
    if flags:                                             # so does the gate's gradient
        assert M.moe_norm_out_backward(n, b.at("a"), None, None, gate, b.at("e"), b.at("f"), None, None, 0,
                                       **kw) == NULL
    # a z that is not read is still checked, and so is everything else beside a missing one
    args = (None, gate, b.at("e"), None, None, None, 0)
    assert M.moe_norm_out_backward(n, b.at("a"), b.at("b") + 4, *args, **kw) == ALIGN
    assert M.moe_norm_out_backward(n, b.at("a"), b.at("e"), *args, **kw) == ALIAS
    assert M.moe_norm_out_backward(n, None, None, *args, **kw) == NULL
    assert M.moe_norm_out_backward(n, b.at("e"), None, *args, **kw) == ALIAS
    assert M.moe_norm_out_backward(n, b.at("a"), None, None, gate, None, None, None, None, 0, **kw) == NULL
    assert b.untouched()
