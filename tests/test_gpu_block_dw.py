"""dw of the norm gradients to the last row, on the GPU.

dw is a sum over all rows, so a bound that grows with the number of rows and
the size of the terms does not see a single row that is lost or counted twice.
Here every term is a whole number: rows of +-1 have rs = 1 (their mean square
is 1, and eps = 2^-126 vanishes beside it), the gradients are +-1, +-2 or +-3,
gates and scales 1, 2 or 4.  A sum of at most 131072 of them stays under 2^24
and is exact in float32 in any order, and each row changes every column."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests.test_gpu_block import DEV, DT, FULL, TOKEN, Gen, Out, workspace

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -126

# a workgroup per row, one to several rows each; a wave per row of 1, 2, 3 and
# 5 chunks; rows that share a wave; eight waves a workgroup; each with rows
# left over, and lengths that cut a chunk or start at odd elements
SHAPES = [(1, 2560), (2, 333), (255, 40), (256, 2560), (257, 2560), (511, 1001), (513, 5120), (1023, 77), (1537, 264),
          (2047, 2560), (2100, 8200), (700, 20480), (600, 40001), (517, 65536),
          (2048, 512), (2049, 520), (2050, 1001), (2051, 1536), (2050, 1600), (2049, 1999), (2050, 2048), (2304, 2560),
          (5003, 2559), (9001, 2560), (2048, 1), (2049, 7), (2063, 16), (4099, 40), (2101, 64), (2055, 65), (4097, 100),
          (2051, 128), (2077, 250), (30001, 128), (50003, 64), (25001, 255),
          (131072, 13), (131071, 64), (65537, 64), (65543, 127), (32771, 250), (32768, 256), (16384, 255), (16391, 333),
          (16385, 512), (40961, 384)]


def whole(g, *shape, values, dtype):
    v = torch.tensor(values, device=DEV, dtype=torch.float32)
    return v[torch.randint(len(values), shape, generator=g.g, device=DEV)].to(dtype)


def column_sums(*factors):
    """The sum over rows of the factors' product, exact in float64."""
    t = factors[0].double()
    for f in factors[1:]:
        t = t * f.double()
    return t.sum(0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_dw_counts_every_row_once(T, H, act):
    dt, g = DT[act], Gen(T, H, act == "f32", 51)
    signs, steps = (-1.0, 1.0), (-3.0, -2.0, -1.0, 1.0, 2.0, 3.0)
    z, dout = whole(g, T, H, values=signs, dtype=dt), whole(g, T, H, values=steps, dtype=dt)
    w = g(H, std=0.2, mean=1.0, dtype=dt)
    norm = M.make_norm(T, H, act, eps=EPS)
    n = Out(T, H, dtype=dt)
    M.moe_norm_in(norm, z, torch.ones_like(w), n.t)
    assert torch.equal(n.t, z)                            # rs is 1
    ws, nb = workspace(norm)
    dx, dw = Out(T, H, dtype=dt), Out(H, dtype=torch.float32)
    M.moe_norm_in_backward(norm, dout, z, w, None, dx.t, dw.t, ws, nb)
    assert torch.equal(dw.t.double(), column_sums(dout, z)) and dw.ok()
    M.moe_norm_in_backward(norm, dout, z, w, dout, dx.t, dw.t, ws, nb)
    assert torch.equal(dw.t.double(), column_sums(dout, z)) and dw.ok()
    for flags in (0, TOKEN, FULL):
        gate, G = None, torch.ones((), device=DEV)
        if flags:
            gate = whole(g, *((T,) if flags == TOKEN else (T, H)), values=(1.0, 2.0, 4.0),
                         dtype=torch.float32 if flags == TOKEN else dt)
            G = gate.reshape(T, -1)
        norm = M.make_norm(T, H, act, eps=EPS, branch_scale=2.0, flags=flags)
        M.moe_norm_out_backward(norm, dout, z, w, gate, dx.t, None, dw.t, ws, nb)
        assert torch.equal(dw.t.double(), 2 * column_sums(dout, z, G)) and dw.ok(), flags
