"""Rows whose last chunks, and slots whose whole row, lie past what the
operators around the routed experts may read: outputs against the 64-bit
definitions (tests/block_ref.py), with NaN where nothing may be read."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests import block_ref as R
from tests.test_gpu_block import DEV, DT, EPS, FLAGS, FULL, NONORM, SIG, TOKEN, Gen, Out, case, run_norm_out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("T,H", [(2050, 2048), (2051, 1600), (2049, 1999), (2048, 1538), (1025, 2048)])
def test_norm_out_chunks_past_the_row(T, H, flags, act):
    """A wave's body holds 1, 2, 3 or 5 chunks a lane: bf16 rows of 193 to 256
    chunks leave the fifth of every lane empty."""
    run_norm_out(T, H, act, flags, nxt=True, residual=T % 2 == 0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(2051, 1600), (3, 33000)])
def test_rows_behind_the_last_chunk_are_not_read(T, H, act):
    """What lies behind a row is the next row: NaN there stays there."""
    dt, g = DT[act], Gen(T, H, 31)
    x, w, dn = g(T, H, dtype=dt), g(H, std=0.1, mean=1.0, dtype=dt), g(T, H, dtype=dt)
    x[1::2] = float("nan")
    norm = M.make_norm(T, H, act, eps=EPS)
    n, dx = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
    M.moe_norm_in(norm, x, w, n.t)
    M.moe_norm_in_backward(norm, dn, x, w, None, dx.t, None, None, 0)
    x, dn = x[::2], dn[::2]
    R.check({"n": n.t[::2]}, R.norm_in(x, w, dtype=dt, eps=EPS, offset=0.0), "norm_in")
    want = R.norm_bwd(dn, x, w, None, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.0, flags=0)
    R.check({"dz": dx.t[::2]}, {"dz": want["dz"]}, "norm_in_backward")
    assert n.t[1::2].isnan().all() and dx.t[1::2].isnan().all() and n.ok() and dx.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [512, 4224, 8192, 16384, 65536])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_dropped_slots_read_nothing(H, bad, act):
    """Row 0 is named only by a dropped pair and holds NaN; rows past 8192
    (float32: 4096) features are several chunks a thread."""
    T, E, k = 260, 8, 2
    g, dt, s, ids, w, row = case(T, H, E, k, 0.0, act)
    y, dout = g(T * k, H, dtype=dt), g(T, H, dtype=dt)
    y[0] = float("nan")
    p = int((row == 0).nonzero())
    t = p // k
    row = row.clone()
    row[p] = bad
    z, out = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
    norm = M.make_norm(T, H, act, eps=EPS, flags=NONORM)
    M.moe_combine_norm(s, norm, y, row, w, None, None, None, None, z.t, out.t, None)
    zr, ez = R.combine(y, row, w, T, k)
    want = R.norm_out(zr, ez, None, None, None, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.0,
                      flags=NONORM)
    R.check({"z": z.t, "out": out.t}, {"z": (zr, ez + zr.abs() * R.u_of(dt)), **want}, "combine_norm")
    dy, dw = Out(T * k, H, dtype=dt, fill=3.0), Out(T, k, dtype=torch.float32)
    old = dy.t.clone()
    M.moe_combine_backward(s, dout, y, row, w, dy.t, dw.t)
    R.check({"dy": dy.t, "dw": dw.t}, R.combine_bwd(dout, y, row, w, old, dtype=dt, dw=True), "combine_backward")
    assert dw.t[t, p % k] == 0 and (dy.t[0] == 3).all()
    dx, dwt = Out(T, H, dtype=dt), Out(T, k, dtype=torch.float32)
    M.moe_dispatch_backward(s, y, row, w, dout, None, dx.t, dwt.t)
    R.check({"dx": dx.t, "dw": dwt.t}, R.dispatch_bwd(y, row, w, dout, None, T, dtype=dt, dw=True), "dispatch")
    M.moe_dispatch_backward(s, y, row, None, None, dout, dx.t, None)
    R.check({"dx": dx.t}, R.dispatch_bwd(y, row, None, None, dout, T, dtype=dt, dw=False), "dispatch, no weights")
    assert all(o.ok() for o in (z, out, dy, dw, dx, dwt))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, TOKEN, FULL, FULL | SIG])
@pytest.mark.parametrize("T,H", [(1, 2560), (5, 77), (2050, 40), (2051, 33), (2051, 1999), (2048, 2560), (3, 9000),
                                 (2, 40000)])
def test_gradient_without_a_norm_needs_no_branch(T, H, flags, act):
    """Without a norm and a gate's gradient nothing depends on z: NULL gives
    the bits of any z."""
    dt, g = DT[act], Gen(T, H, flags, 37)
    dout, z = g(T, H, dtype=dt), g(T, H, dtype=dt)
    gate = g(T) if flags & TOKEN else g(T, H, dtype=dt) if flags else None
    norm = M.make_norm(T, H, act, branch_scale=1.25, flags=flags | NONORM)
    a, b = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
    M.moe_norm_out_backward(norm, dout, z, None, gate, a.t, None, None, None, 0)
    M.moe_norm_out_backward(norm, dout, None, None, gate, b.t, None, None, None, 0)
    assert torch.equal(a.t, b.t) and a.t.isfinite().all() and a.ok() and b.ok()
