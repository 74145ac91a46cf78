"""moe_router_backward: an output has the same bits whichever of the others are
asked for, whether one launch or two make them."""
import itertools

import pytest
import torch

from tests.test_gpu_train import RouterCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k", [
    (1, 128, 3, 3), (200, 256, 12, 4), (333, 384, 60, 10), (257, 640, 33, 16),   # one launch for both products
    (90, 256, 40, 17),                                                          # more slots than it takes
    (2100, 2560, 64, 5),                                                        # more gathered bytes
    (3000, 128, 4, 3), (4096, 128, 2, 2)])                                      # more pairs per expert
def test_bits_do_not_depend_on_what_is_wanted(T, H, E, k, act):
    c = RouterCase(T, H, E, k, act, seed=23)
    c.call()
    c.check(f"router {T} {H} {E} {k} {act}")
    want = {n: v.clone() for n, v in c.got().items()}
    for on in itertools.product((True, False), repeat=3):
        if not any(on):
            continue
        for o in (c.dx, c.dwr, c.db):
            o.t.fill_(77)
        c.call(*on)
        for asked, (n, v) in zip(on, c.got().items()):
            assert torch.equal(v, want[n]) if asked else bool((v == 77).all()), (on, n)
        assert c.dx.ok() and c.dwr.ok() and c.db.ok()
