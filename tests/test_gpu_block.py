"""The operators around the routed experts on the GPU against their 64-bit
definitions (tests/block_ref.py), at the sizes, strides of work and special
values where they can go wrong."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests import block_ref as R

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
GUARD = 64
TOKEN, FULL, SIG, NONORM = R.GATE_TOKEN, R.GATE_FULL, R.SIGMOID, R.NO_NORM


class Gen:
    def __init__(self, *key):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(hash(key) % (1 << 31))

    def __call__(self, *shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std + mean).to(dtype)


class Out:
    """An output tensor with a guard of sentinels behind it."""

    def __init__(self, *shape, dtype, fill=float("nan")):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + GUARD,), -77.0, dtype=dtype, device=DEV)
        self.t = self.buf[:n].view(*shape)
        self.t.fill_(fill)

    def ok(self):
        return bool((self.buf[self.t.numel():] == -77.0).all())


def workspace(norm):
    n = M.moe_norm_workspace_size(norm)
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device=DEV), n


def run_norm_in(T, H, act, offset=0.0, x=None, w=None, seed=0, bwd=True, dres=True, rscale=1.0):
    g, dt = Gen(T, H, act == "f32", seed), DT[act]
    x = g(T, H, dtype=dt) if x is None else x
    w = g(H, std=0.2, mean=1.0 - offset, dtype=dt) if w is None else w
    norm = M.make_norm(T, H, act, eps=EPS, weight_offset=offset, residual_scale=rscale)
    n = Out(T, H, dtype=dt)
    M.moe_norm_in(norm, x, w, n.t)
    R.check({"n": n.t}, R.norm_in(x, w, dtype=dt, eps=EPS, offset=offset), f"norm_in {T}x{H} {act}")
    assert n.ok()
    if not bwd:
        return
    dn, dr = g(T, H, std=0.5, dtype=dt), g(T, H, std=0.5, dtype=dt) if dres else None
    dx, dw = Out(T, H, dtype=dt), Out(H, dtype=torch.float32)
    ws, nb = workspace(norm)
    M.moe_norm_in_backward(norm, dn, x, w, dr, dx.t, dw.t, ws, nb)
    want = R.norm_bwd(dn, x, w, None, dr, dtype=dt, eps=EPS, offset=offset, rscale=rscale, bscale=1.0,
                      flags=0)
    R.check({"dz": dx.t, "dw": dw.t}, want, f"norm_in_backward {T}x{H} {act}")
    assert dx.ok() and dw.ok()
    # without dw: the same dx, no workspace
    dx2 = Out(T, H, dtype=dt)
    M.moe_norm_in_backward(norm, dn, x, w, dr, dx2.t, None, None, 0)
    assert torch.equal(dx.t, dx2.t) and dx2.ok()


# one element to the widest rows, on both sides of every power that a lane,
# wave or workgroup covers, and lengths that no vector divides
WIDTHS = [1, 2, 3, 7, 8, 9, 31, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 1001, 1024, 1029, 1536, 2047,
          2048, 2049, 2560, 4095, 4096, 4097, 5120, 8192, 8200, 16384, 16390, 32768, 65535, 65536]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_in_widths(H, act):
    run_norm_in(5, H, act, offset=1.0 if H % 2 else 0.0, dres=H % 3 != 0, rscale=0.5)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 2560), (2, 2560), (3, 40), (4, 2560), (63, 333), (64, 2560), (65, 129),
                                 (511, 256), (513, 520), (1023, 96), (1025, 2560), (2049, 64), (4099, 33)])
def test_norm_in_rows(T, H, act):
    run_norm_in(T, H, act)


def run_norm_out(T, H, act, flags, nxt=True, residual=True, offset=0.0, rscale=0.75, bscale=1.25, seed=0,
                 grads=True):
    g, dt = Gen(T, H, act == "f32", flags, seed), DT[act]
    z = g(T, H, std=0.3, dtype=dt)
    w = None if flags & NONORM else g(H, std=0.2, mean=1.0 - offset, dtype=dt)
    gate = g(T) if flags & TOKEN else g(T, H, dtype=dt) if flags & FULL else None
    res = g(T, H, dtype=dt) if residual else None
    wn = g(H, std=0.2, mean=1.0 - offset, dtype=dt) if nxt else None
    norm = M.make_norm(T, H, act, eps=EPS, weight_offset=offset, residual_scale=rscale,
                       branch_scale=bscale, flags=flags)
    kw = dict(dtype=dt, eps=EPS, offset=offset, rscale=rscale, bscale=bscale, flags=flags)
    what = f"norm_out {T}x{H} {act} flags {flags}"
    out, nn = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
    M.moe_norm_out(norm, z, w, gate, res, wn, out.t, nn.t if nxt else None)
    R.check({"out": out.t, "n_next": nn.t},
            R.norm_out(z.double(), torch.zeros_like(z, dtype=torch.float64), w, gate, res, wn, **kw), what)
    assert out.ok() and nn.ok()
    dout = g(T, H, std=0.5, dtype=dt)
    dz = Out(T, H, dtype=dt)
    dg = None
    if gate is not None and grads:
        dg = Out(*gate.shape, dtype=gate.dtype)
    dw = Out(H, dtype=torch.float32) if w is not None and grads else None
    ws, nb = workspace(norm)
    M.moe_norm_out_backward(norm, dout, z, w, gate, dz.t, dg.t if dg else None, dw.t if dw else None,
                            ws if dw else None, nb if dw else 0)
    want = R.norm_bwd(dout, z, w, gate, None, **kw)
    got = {"dz": dz.t, "dw": dw.t if dw else None, "dgate": dg.t if dg else None}
    got = {n: v for n, v in got.items() if v is not None}
    R.check(got, {n: want[n] for n in got}, what + " backward")
    assert dz.ok() and (dw is None or dw.ok()) and (dg is None or dg.ok())


FLAGS = [0, TOKEN, FULL, TOKEN | SIG, FULL | SIG, NONORM, NONORM | TOKEN, NONORM | FULL | SIG]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("T,H", [(1, 2560), (6, 77), (37, 1288), (700, 264), (9, 6144)])
def test_norm_out(T, H, flags, act):
    run_norm_out(T, H, act, flags, nxt=T % 2 == 1, residual=H != 264, offset=1.0 if H == 77 else 0.0)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("T,H", [(1024, 520), (2048, 8), (2050, 1001), (2051, 1536), (2304, 2560),
                                 (2049, 2561), (4097, 33), (2050, 1280), (2050, 257)])
def test_norm_out_many_rows(T, H, flags, act):
    """From 1024 (2048) rows on a row is one wave's work."""
    run_norm_out(T, H, act, flags, nxt=H % 2 == 0, residual=H != 520)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("T,H", [(2048, 1), (1025, 3), (2049, 7), (2063, 16), (2050, 31), (4099, 40), (2101, 64),
                                 (2055, 65), (4097, 100), (2051, 128), (2049, 129), (2077, 250), (2049, 256),
                                 (30001, 128), (50003, 64), (25001, 255)])
def test_norm_out_rows_that_share_a_wave(T, H, flags, act):
    run_norm_out(T, H, act, flags, nxt=T % 2 == 1, residual=H != 65)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, TOKEN, FULL | SIG])
@pytest.mark.parametrize("T,H", [(131072, 13), (65537, 64), (32771, 250), (16384, 255), (16391, 333), (16385, 512)])
def test_norm_out_eight_waves(T, H, flags, act):
    """Rows enough for the gradient's larger workgroups."""
    run_norm_out(T, H, act, flags, nxt=False, residual=False)


def test_special_values_stay_with_their_row_in_a_shared_wave():
    T, H = 2050, 40
    g = Gen(T, H)
    for act in ("bf16", "f32"):
        dt = DT[act]
        x, w, dn = g(T, H, dtype=dt), g(H, std=0.1, mean=1.0, dtype=dt), g(T, H, dtype=dt)
        bad = [3, 1029, 2049]
        clean = x.clone()
        for i, r in enumerate(bad):
            x[r, i] = float("nan") if i else float("inf")
        keep = [r for r in range(T) if r not in bad]
        norm = M.make_norm(T, H, act, eps=EPS)
        n, dx = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
        M.moe_norm_in(norm, x, w, n.t)
        M.moe_norm_in_backward(norm, dn, x, w, None, dx.t, None, None, 0)
        v, b = R.norm_in(clean, w, dtype=dt, eps=EPS, offset=0.0)["n"]
        R.check({"n": n.t[keep]}, {"n": (v[keep], b[keep])}, "shared wave")
        v, b = R.norm_bwd(dn, clean, w, None, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.0,
                          flags=0)["dz"]
        R.check({"dz": dx.t[keep]}, {"dz": (v[keep], b[keep])}, "shared wave backward")
        assert n.t[bad[1:]].isnan().all() and dx.t[bad[1:]].isnan().all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 5, 8, 63, 512, 513, 1537, 2049, 4100, 8192, 8201, 20480, 65535, 65536])
def test_norm_out_widths(H, act):
    run_norm_out(4, H, act, FULL | SIG)
    run_norm_out(3, H, act, TOKEN, grads=False)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 2, 6, 7, 333, 2560, 2563, 8194, 20485, 65535])
def test_norm_out_single_row(H, act):
    """One row is its own sum of columns."""
    run_norm_out(1, H, act, FULL)
    run_norm_out(1, H, act, TOKEN | SIG, nxt=False)


# ---------------------------------------------------------------------------
# Sorted rows
# ---------------------------------------------------------------------------


def routes(g, T, E, k, drop=0.0, skew=0.0):
    logits = g(T, E) - skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    top, ids = logits.topk(k, dim=1)
    order = ids.reshape(-1).argsort(stable=True)
    row = torch.empty(T * k, dtype=torch.int32, device=DEV)
    row[order] = torch.arange(T * k, device=DEV, dtype=torch.int32)
    if drop:
        off = torch.rand(T * k, generator=g.g, device=DEV)
        row[off < drop] = -1
        row[off < drop / 2] = T * k           # past the end: dropped as well
    return ids.to(torch.int32), torch.softmax(top, 1), row


ROUTES = [  # T, H, E, k, drop
    (1, 128, 1, 1, 0.0), (1, 2560, 512, 10, 0.0), (3, 384, 5, 5, 0.0), (8, 2560, 512, 10, 0.3),
    (16, 256, 16, 2, 0.0), (33, 640, 60, 3, 0.5), (17, 1152, 40, 17, 0.0), (257, 128, 33, 7, 0.1),
    (40, 8192, 64, 8, 0.0), (5, 128, 1024, 130, 0.2), (700, 256, 512, 10, 0.0), (4, 65536, 8, 2, 0.0),
    (9, 512, 8, 4, 1.1),                      # every pair dropped
    (1100, 4096, 64, 16, 0.1),                # rows past 128 MiB
    (2, 8192, 1024, 1024, 0.1),               # every expert, 64 KB of LDS for the dot products
]
RID = [f"{t}x{h}-{e}-{k}-{d}" for t, h, e, k, d in ROUTES]


def case(T, H, E, k, drop, act):
    g, dt = Gen(T, H, E, k, act == "f32"), DT[act]
    ids, w, row = routes(g, T, E, k, drop, skew=0.5)
    return g, dt, M.make_shape(T, H, E, 128, k, act), ids, w, row


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,drop", ROUTES, ids=RID)
def test_dispatch(T, H, E, k, drop, act):
    g, dt, s, _, w, row = case(T, H, E, k, drop, act)
    x, drows, add = g(T, H, dtype=dt), g(T * k, H, std=0.5, dtype=dt), g(T, H, dtype=dt)
    for weights in (None, w):
        rows = Out(T * k, H, dtype=dt, fill=3.0)
        old = rows.t.clone()
        M.moe_dispatch(s, x, row, weights, rows.t)
        R.check({"rows": rows.t}, R.dispatch(x, row, weights, old, dtype=dt), "dispatch")
        assert rows.ok()
        for dx_in in (None, add):
            dx = Out(T, H, dtype=dt)
            dw = Out(T, k, dtype=torch.float32) if weights is not None else None
            M.moe_dispatch_backward(s, drows, row, weights, x if dw else None, dx_in, dx.t,
                                    dw.t if dw else None)
            want = R.dispatch_bwd(drows, row, weights, x, dx_in, T, dtype=dt, dw=dw is not None)
            R.check({"dx": dx.t, "dw": dw.t if dw else None}, want, "dispatch_backward")
            assert dx.ok() and (dw is None or dw.ok())
    # weights without their gradient
    dx2 = Out(T, H, dtype=dt)
    M.moe_dispatch_backward(s, drows, row, w, None, add, dx2.t, None)
    R.check({"dx": dx2.t}, R.dispatch_bwd(drows, row, w, x, add, T, dtype=dt, dw=False), "no dw")


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(256, 5504), (257, 4224), (300, 5504), (258, 7168), (261, 2176)])
def test_dispatch_backward_in_rounds(T, H, act):
    """Past 256 tokens a long row is a workgroup's work in rounds."""
    k = 3
    g, dt, s, _, w, row = case(T, H, 40, k, 0.1, act)
    x, drows, dx_in = g(T, H, dtype=dt), g(T * k, H, std=0.5, dtype=dt), g(T, H, dtype=dt)
    dx, dw = Out(T, H, dtype=dt), Out(T, k, dtype=torch.float32)
    M.moe_dispatch_backward(s, drows, row, w, x, dx_in, dx.t, dw.t)
    want = R.dispatch_bwd(drows, row, w, x, dx_in, T, dtype=dt, dw=True)
    R.check({"dx": dx.t, "dw": dw.t}, want, "dispatch_backward")
    assert dx.ok() and dw.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,drop", ROUTES, ids=RID)
def test_combine_and_route_backward(T, H, E, k, drop, act):
    g, dt, s, ids, w, row = case(T, H, E, k, drop, act)
    dout, y = g(T, H, std=0.5, dtype=dt), g(T * k, H, dtype=dt)
    dy, dw = Out(T * k, H, dtype=dt, fill=3.0), Out(T, k, dtype=torch.float32)
    old = dy.t.clone()
    M.moe_combine_backward(s, dout, y, row, w, dy.t, dw.t)
    R.check({"dy": dy.t, "dw": dw.t}, R.combine_bwd(dout, y, row, w, old, dtype=dt, dw=True),
            "combine_backward")
    dy2 = Out(T * k, H, dtype=dt, fill=3.0)
    M.moe_combine_backward(s, dout, None, row, w, dy2.t, None)
    assert torch.equal(dy.t, dy2.t) and dy.ok() and dw.ok() and dy2.ok()
    g_w, dl = g(T, k), Out(T, E, dtype=torch.float32)
    M.moe_route_backward(s, ids, w, g_w, dl.t)
    R.check({"dlogits": dl.t}, R.route_bwd(ids, w, g_w, E), "route_backward")
    assert dl.ok()
    if k > 1:                                  # an id out of range is left out
        ids = ids.clone()
        ids[:, 1] = torch.where(torch.arange(T, device=DEV) % 2 == 0, -1, E).to(torch.int32)
        M.moe_route_backward(s, ids, w, g_w, dl.t)
        R.check({"dlogits": dl.t}, R.route_bwd(ids, w, g_w, E), "route_backward, bad ids")
        assert dl.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,drop", ROUTES, ids=RID)
def test_combine_norm(T, H, E, k, drop, act):
    g, dt, s, _, w, row = case(T, H, E, k, drop, act)
    y = g(T * k, H, dtype=dt)
    for flags, nxt, residual, keep in ((0, True, True, True), (NONORM, True, True, False),
                                       (FULL | SIG, False, True, False), (TOKEN, True, False, True)):
        wp = None if flags & NONORM else g(H, std=0.2, mean=1.0, dtype=dt)
        gate = g(T) if flags & TOKEN else g(T, H, dtype=dt) if flags & FULL else None
        res = g(T, H, dtype=dt) if residual else None
        wn = g(H, std=0.2, mean=1.0, dtype=dt) if nxt else None
        norm = M.make_norm(T, H, act, eps=EPS, residual_scale=0.75, branch_scale=1.25, flags=flags)
        z, out, nn = (Out(T, H, dtype=dt) for _ in range(3))
        M.moe_combine_norm(s, norm, y, row, w, wp, gate, res, wn, z.t if keep else None, out.t,
                           nn.t if nxt else None)
        zr, ez = R.combine(y, row, w, T, k)
        want = R.norm_out(zr, ez, wp, gate, res, wn, dtype=dt, eps=EPS, offset=0.0, rscale=0.75,
                          bscale=1.25, flags=flags)
        if keep:
            want["z"] = (zr, ez + zr.abs() * R.u_of(dt))
        R.check({"z": z.t, "out": out.t, "n_next": nn.t}, want, f"combine_norm flags {flags}")
        assert z.ok() and out.ok() and nn.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k", [(7, 2560, 64, 10), (50, 384, 16, 3), (3, 4096, 32, 20)])
def test_bits_shared_with_combine(T, H, E, k, act):
    """moe_combine_norm without norm, gate and scales is moe_combine; the
    unweighted dispatch gradient is the combine with weights of one."""
    g, dt, s, _, w, row = case(T, H, E, k, 0.0, act)
    y, res = g(T * k, H, dtype=dt), g(T, H, dtype=dt)
    ref, out = Out(T, H, dtype=dt), Out(T, H, dtype=dt)
    M.moe_combine(s, y, row, w, res, ref.t)
    M.moe_combine_norm(s, M.make_norm(T, H, act, flags=NONORM), y, row, w, None, None, res, None, None,
                       out.t, None)
    assert torch.equal(ref.t, out.t)
    M.moe_combine(s, y, row, torch.ones_like(w), res, ref.t)
    M.moe_dispatch_backward(s, y, row, None, None, res, out.t, None)
    assert torch.equal(ref.t, out.t)


# ---------------------------------------------------------------------------
# Special values, empty batches, far offsets
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H", [40, 2560, 2561, 9000])
def test_special_rows_stay_in_their_row(H, act):
    dt, g, T = DT[act], Gen(H, 5), 9
    x, w = g(T, H, dtype=dt), g(H, std=0.1, mean=1.0, dtype=dt)
    clean = x.clone()
    x[1] = 0.0
    x[3, H // 2] = float("nan")
    x[5, H - 1] = float("inf")
    x[7] = torch.finfo(dt).tiny
    clean[1], clean[7] = x[1], x[7]
    norm = M.make_norm(T, H, act, eps=EPS)
    n = Out(T, H, dtype=dt)
    M.moe_norm_in(norm, x, w, n.t)
    keep = [0, 1, 2, 4, 6, 7, 8]
    v, b = R.norm_in(clean, w, dtype=dt, eps=EPS, offset=0.0)["n"]
    R.check({"n": n.t[keep]}, {"n": (v[keep], b[keep])}, "special rows")
    assert (n.t[1] == 0).all()
    assert n.t[3].isnan().all()
    assert n.t[5, H - 1].isnan() and (n.t[5, :H - 1] == 0).all()
    dn, dx, dw = g(T, H, dtype=dt), Out(T, H, dtype=dt), Out(H, dtype=torch.float32)
    ws, nb = workspace(norm)
    M.moe_norm_in_backward(norm, dn, x, w, None, dx.t, dw.t, ws, nb)
    v, b = R.norm_bwd(dn, clean, w, None, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.0,
                      flags=0)["dz"]
    R.check({"dz": dx.t[keep]}, {"dz": (v[keep], b[keep])}, "special rows backward")
    assert dx.t[3].isnan().all() and dw.t.isnan().all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("flags", [0, TOKEN, FULL | SIG])
@pytest.mark.parametrize("T,H", [(5, 40), (2050, 77), (2051, 2560), (3, 9000), (2, 33000)])
def test_gradient_without_a_norm_does_not_hold_the_branch(T, H, flags, act):
    """dz = G db: infinity and NaN in z reach the gate's gradient only."""
    dt, g = DT[act], Gen(T, H, 7)
    z, dout = g(T, H, dtype=dt), g(T, H, dtype=dt)
    gate = g(T) if flags & TOKEN else g(T, H, dtype=dt) if flags else None
    norm = M.make_norm(T, H, act, eps=EPS, branch_scale=1.25, flags=flags | NONORM)
    v, b = R.norm_bwd(dout, z, None, gate, None, dtype=dt, eps=EPS, offset=0.0, rscale=1.0, bscale=1.25,
                      flags=flags | NONORM)["dz"]
    z[0, H // 2], z[1, H - 1] = float("inf"), float("nan")
    for wanted in (True, False):
        dz = Out(T, H, dtype=dt)
        dg = Out(*gate.shape, dtype=gate.dtype) if wanted and flags else None
        M.moe_norm_out_backward(norm, dout, z, None, gate, dz.t, dg.t if dg else None, None, None, 0)
        R.check({"dz": dz.t}, {"dz": (v, b)}, "no norm")
        assert dz.ok()
        if dg:
            bad = [0, 1] if flags & TOKEN else [(0, H // 2), (1, H - 1)]
            assert not any(dg.t[i].isfinite() for i in bad) and dg.t[2:].isfinite().all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_dropped_pairs_are_not_read(act):
    """Rows that only a dropped pair would name may hold anything; a NaN in a
    kept row stays with its token."""
    T, H, E, k = 6, 512, 8, 2
    g, dt, s, ids, w, row = case(T, H, E, k, 0.0, act)
    y, dout = g(T * k, H, dtype=dt), g(T, H, dtype=dt)
    dead = row[2 * k].item()                     # token 2, slot 0
    y[dead] = float("nan")
    row = row.clone()
    row[2 * k] = -1
    norm = M.make_norm(T, H, act, eps=EPS, flags=NONORM)
    out = Out(T, H, dtype=dt)
    M.moe_combine_norm(s, norm, y, row, w, None, None, None, None, None, out.t, None)
    assert out.t.isfinite().all()
    dy, dw = Out(T * k, H, dtype=dt, fill=3.0), Out(T, k, dtype=torch.float32)
    M.moe_combine_backward(s, dout, y, row, w, dy.t, dw.t)
    assert dw.t.isfinite().all() and dw.t[2, 0] == 0 and (dy.t[dead] == 3.0).all()
    dx = Out(T, H, dtype=dt)
    M.moe_dispatch_backward(s, y, row, w, dout, None, dx.t, dw.t)
    assert dx.t.isfinite().all() and dw.t.isfinite().all() and dw.t[2, 0] == 0
    y[row[5 * k + 1].item()] = float("inf")
    M.moe_combine_norm(s, norm, y, row, w, None, None, None, None, None, out.t, None)
    assert out.t[:5].isfinite().all() and out.t[5].isinf().all()


def test_empty_batch_writes_zero_dw():
    norm = M.make_norm(0, 300, "bf16")
    e = torch.empty(0, 300, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(300, dtype=torch.bfloat16, device=DEV)
    dw = Out(300, dtype=torch.float32)
    M.moe_norm_in_backward(norm, e, e, w, None, e, dw.t, None, 0)
    assert (dw.t == 0).all() and dw.ok()
    dw.t.fill_(5)
    M.moe_norm_out_backward(norm, e, e, w, None, e, None, dw.t, None, 0)
    assert (dw.t == 0).all() and dw.ok()
    M.moe_norm_in(norm, e, w, e)


def _pick(t, rows):
    return t[rows].contiguous()


def test_norm_offsets_past_32_bits():
    """T * H * 2 bytes past 2^32: the last rows are read and written at their
    place."""
    T, H = 70001, 32776
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=Gen(1).g)
    assert x.numel() > 1 << 31
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    norm = M.make_norm(T, H, "bf16", eps=EPS)
    n = torch.empty_like(x)
    M.moe_norm_in(norm, x, w, n)
    rows = torch.tensor([0, 1, 32767, 65521, 65535, 65536, T - 2, T - 1], device=DEV)
    R.check({"n": _pick(n, rows)}, R.norm_in(_pick(x, rows), w, dtype=torch.bfloat16, eps=EPS, offset=0.0),
            "far rows")
    dx = torch.empty_like(x)
    M.moe_norm_in_backward(norm, n, x, w, None, dx, None, None, 0)
    want = R.norm_bwd(_pick(n, rows), _pick(x, rows), w, None, None, dtype=torch.bfloat16, eps=EPS,
                      offset=0.0, rscale=1.0, bscale=1.0, flags=0)
    R.check({"dz": _pick(dx, rows)}, {"dz": want["dz"]}, "far rows backward")


def test_rows_past_32_bits():
    """P * H past 2^32 elements: 70000 tokens in 16 slots of 4096 features."""
    T, H, E, k = 70000, 4096, 32, 16
    g = Gen(2)
    s = M.make_shape(T, H, E, 128, k, "bf16")
    P = T * k
    assert P * H > 1 << 32
    row = torch.randperm(P, generator=g.g, device=DEV).to(torch.int32)
    w = torch.rand(T, k, generator=g.g, device=DEV)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g.g)
    rows = torch.empty(P, H, dtype=torch.bfloat16, device=DEV)
    M.moe_dispatch(s, x, row, None, rows)
    tok = torch.tensor([0, 1, 4095, 34999, T - 1], device=DEV)
    r = row.view(T, k)[tok].long()
    assert torch.equal(rows[r.reshape(-1)], x[tok].repeat_interleave(k, 0))
    dy, dw = torch.empty_like(rows), torch.empty(T, k, device=DEV)
    M.moe_combine_backward(s, x, rows, row, w, dy, dw)
    want = (x[tok].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    assert ((dw[tok].double() - want).abs() <= want * (R.chain(H) + 2) * R.E).all()
    exp = x[tok].double()[:, None] * w[tok].double()[:, :, None]
    got = dy[r.reshape(-1)].view(len(tok), k, H).double()
    assert ((got - exp).abs() <= exp.abs() * (R.E + R.u_of(torch.bfloat16)) + R.TINY).all()
    dx = torch.empty_like(x)
    M.moe_dispatch_backward(s, rows, row, None, None, None, dx, None)
    exp = k * x[tok].double()
    assert ((dx[tok].double() - exp).abs() <= exp.abs() * ((k + 1) * R.E + R.u_of(torch.bfloat16))).all()
    norm = M.make_norm(T, H, "bf16", eps=EPS, flags=NONORM)
    M.moe_combine_norm(s, norm, rows, row, w, None, None, None, None, None, dx, None)
    exp = x[tok].double() * w[tok].double().sum(1, keepdim=True)
    assert ((dx[tok].double() - exp).abs() <= exp.abs() * ((2 * k + 2) * R.E + R.u_of(torch.bfloat16))).all()


# ---------------------------------------------------------------------------
# Together, as a program uses them
# ---------------------------------------------------------------------------


class Block:
    """One float32 block around torch's own expert products: norm, route,
    dispatch, experts, combine with the norm after it, residual, next norm;
    then the gradients of everything."""

    def __init__(self, T=48, H=256, E=16, k=2, act="f32"):
        g, dt = Gen(T, H, E, k, 9), DT[act]
        self.dims, self.act = (T, H, E, k), act
        self.x = g(T, H, dtype=dt)
        self.wr = g(E, H, std=0.05, dtype=dt)
        self.we = g(E, H, H, std=0.05, dtype=dt)
        self.w1, self.w2, self.w3 = (g(H, std=0.1, mean=1.0, dtype=dt) for _ in range(3))
        self.gate = g(T)
        self.d_out, self.d_next = g(T, H, dtype=dt), g(T, H, dtype=dt)
        self.buf = M.MoELayerBuffers(T, H, E, 128, k, act, device=DEV)
        self.pre = M.make_norm(T, H, act, eps=EPS)
        self.post = M.make_norm(T, H, act, eps=EPS, residual_scale=0.9, branch_scale=1.1,
                                flags=TOKEN | SIG)
        self.nxt = M.make_norm(T, H, act, eps=EPS)
        self.back = M.make_norm(T, H, act, eps=EPS, residual_scale=0.9)
        new = lambda *s, d=dt: torch.zeros(s, dtype=d, device=DEV)
        P = T * k
        self.n, self.z, self.out, self.n_next = (new(T, H) for _ in range(4))
        self.rows, self.drows, self.dy = new(P, H), new(P, H), new(P, H)
        self.dv, self.dz, self.dn, self.dx = (new(T, H) for _ in range(4))
        self.dgate, self.dw1, self.dw2, self.dw3 = (new(m, d=torch.float32) for m in (T, H, H, H))
        self.dtopk, self.dlogits = new(T, k, d=torch.float32), new(T, E, d=torch.float32)
        self.ws, self.nb = workspace(self.pre)

    def experts(self, rows, transpose=False):
        T, H, E, k = self.dims
        e = self.buf.topk_ids.reshape(-1)[self.buf.sorted_pair.long()].long()
        w = self.we[e]
        w = w.transpose(1, 2) if transpose else w
        return (w * rows[:, None, :]).sum(2)          # y = W x, or W^T dy

    def forward(self):
        b = self.buf
        M.moe_norm_in(self.pre, self.x, self.w1, self.n)
        b.route_permute(self.n, self.wr)
        M.moe_dispatch(b.shape, self.n, b.pair_row, None, self.rows)
        self.y = self.experts(self.rows)
        M.moe_combine_norm(b.shape, self.post, self.y, b.pair_row, b.topk_w, self.w2, self.gate, self.x,
                           self.w3, self.z, self.out, self.n_next)

    def backward(self):
        b = self.buf
        M.moe_norm_in_backward(self.nxt, self.d_next, self.out, self.w3, self.d_out, self.dv, self.dw3,
                               self.ws, self.nb)
        M.moe_norm_out_backward(self.post, self.dv, self.z, self.w2, self.gate, self.dz, self.dgate,
                                self.dw2, self.ws, self.nb)
        M.moe_combine_backward(b.shape, self.dz, self.y, b.pair_row, b.topk_w, self.dy, self.dtopk)
        M.moe_route_backward(b.shape, b.topk_ids, b.topk_w, self.dtopk, self.dlogits)
        self.drows.copy_(self.experts(self.dy, transpose=True))
        router = (self.dlogits[:, :, None] * self.wr[None].float()).sum(1).to(self.x.dtype)
        M.moe_dispatch_backward(b.shape, self.drows, b.pair_row, None, None, router, self.dn, None)
        M.moe_norm_in_backward(self.back, self.dn, self.x, self.w1, self.dv, self.dx, self.dw1, self.ws,
                               self.nb)

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("n", "out", "n_next", "dx", "dw1", "dw2", "dw3",
                                                      "dgate", "dlogits", "dy", "dn")}


def test_block_gradients_match_autograd():
    """The chain of calls against torch's differentiation of the whole block in
    float64 for the same routes.  Each of the ten stages is off by at most
    (H / 64 + 60) 2^-24 = 4e-6 of the magnitudes it adds, and no sum here
    cancels by more than a factor of ten in the norm of the whole output:
    2e-4 relative in norm."""
    b = Block()
    T, H, E, k = b.dims
    b.forward()
    b.backward()
    D = {n: getattr(b, n).double().requires_grad_() for n in ("x", "w1", "w2", "w3", "gate", "wr")}
    nrm = lambda v, w: v * ((v * v).mean(1, keepdim=True) + EPS) ** -0.5 * w
    n = nrm(D["x"], D["w1"])
    n.retain_grad()
    logits = n @ D["wr"].t()
    logits.retain_grad()
    ids = b.buf.topk_ids.long()
    w = torch.softmax(logits.gather(1, ids), 1)
    ys = (b.we.double()[ids] * n[:, None, None, :]).sum(3)           # [T][k][H]
    z = (w[:, :, None] * ys).sum(1)
    v = 0.9 * D["x"] + 1.1 * torch.sigmoid(D["gate"])[:, None] * nrm(z, D["w2"])
    nn = nrm(v, D["w3"])
    ((v * b.d_out.double()).sum() + (nn * b.d_next.double()).sum()).backward()
    rel = lambda a, r: float((a.double() - r).norm() / r.norm())
    for name, got, want in (("n", b.n, n), ("out", b.out, v), ("n_next", b.n_next, nn),
                            ("dx", b.dx, D["x"].grad), ("dw1", b.dw1, D["w1"].grad),
                            ("dw2", b.dw2, D["w2"].grad), ("dw3", b.dw3, D["w3"].grad),
                            ("dgate", b.dgate, D["gate"].grad), ("dlogits", b.dlogits, logits.grad),
                            ("dn", b.dn, n.grad)):
        assert rel(got, want.detach()) <= 2e-4, (name, rel(got, want.detach()))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_block_in_a_graph_repeats(act):
    """Captured once, replayed with eager work and new inputs in between: every
    replay has the bits of the eager run on the same inputs."""
    b = Block(act=act)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    b.y = b.y.clone()
    y, drows = b.y, b.drows

    def calls():
        bf = b.buf
        M.moe_norm_in(b.pre, b.x, b.w1, b.n)
        bf.route_permute(b.n, b.wr)
        M.moe_dispatch(bf.shape, b.n, bf.pair_row, None, b.rows)
        M.moe_combine_norm(bf.shape, b.post, y, bf.pair_row, bf.topk_w, b.w2, b.gate, b.x, b.w3, b.z,
                           b.out, b.n_next)
        M.moe_norm_in_backward(b.nxt, b.d_next, b.out, b.w3, b.d_out, b.dv, b.dw3, b.ws, b.nb)
        M.moe_norm_out_backward(b.post, b.dv, b.z, b.w2, b.gate, b.dz, b.dgate, b.dw2, b.ws, b.nb)
        M.moe_combine_backward(bf.shape, b.dz, y, bf.pair_row, bf.topk_w, b.dy, b.dtopk)
        M.moe_route_backward(bf.shape, bf.topk_ids, bf.topk_w, b.dtopk, b.dlogits)
        M.moe_dispatch_backward(bf.shape, drows, bf.pair_row, None, None, None, b.dn, None)
        M.moe_norm_in_backward(b.back, b.dn, b.x, b.w1, b.dv, b.dx, b.dw1, b.ws, b.nb)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        b.x.copy_(Gen(i, 77)(*b.x.shape, dtype=b.x.dtype))
        calls()
        torch.cuda.synchronize()
        want = b.outputs()
        for n in want:
            getattr(b, n).fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = b.outputs()
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


@pytest.mark.parametrize("T,H,E,I,k,tiled", [(8, 512, 64, 128, 6, True), (40, 256, 16, 64, 2, False)])
def test_layer_buffers_block(T, H, E, I, k, tiled):
    """MoELayerBuffers.block: norm, routed layer and residual have the bits of
    moe_norm_in + moe_layer; the next block starts from its n_next."""
    g, bf = Gen(T, H, 21), torch.bfloat16
    buf = M.MoELayerBuffers(T, H, E, I, k, device=DEV, tiled=tiled)
    wr = g(E, H, std=0.05, dtype=bf)
    ws = [g(E, *sh, std=0.05, dtype=bf) for sh in ((I, H), (I, H), (H, I))]
    ex = M.make_experts(*ws)
    if tiled:
        dst = [torch.empty_like(w) for w in ws]
        M.moe_tile_experts(M.make_shape(T, H, E, I, k), ex, M.make_experts(*dst))
        ex = M.make_experts(*dst)
    w1, w2 = g(H, std=0.1, mean=1.0, dtype=bf), g(H, std=0.1, mean=1.0, dtype=bf)
    x = g(T, H, dtype=bf)
    pre, post = M.make_norm(T, H, eps=EPS), M.make_norm(T, H, eps=EPS, flags=NONORM)
    n, out, n_next, ref = (Out(T, H, dtype=bf) for _ in range(4))
    buf.block(x, pre, w1, wr, None, ex, post, None, residual=x, w_next=w2, n=n.t, out=out.t, n_next=n_next.t)
    ids = buf.topk_ids.clone()
    M.moe_norm_in(pre, x, w1, ref.t)
    assert torch.equal(n.t, ref.t)
    other = M.MoELayerBuffers(T, H, E, I, k, device=DEV, tiled=tiled)
    other.layer(n.t, wr, None, ex, residual=x)
    assert torch.equal(ids, other.topk_ids) and torch.equal(out.t, other.out)
    # n_next is the norm of the sum before its rounding to out
    v = out.t.double()
    want, err = R._norm(v, v.abs() * R.u_of(bf), w2.double(), EPS)
    R.check({"n": n_next.t}, {"n": (want, err + want.abs() * R.u_of(bf) + R.TINY)}, "n_next")
    out2 = Out(T, H, dtype=bf)
    buf.block(None, None, None, wr, None, ex, post, None, residual=out.t, n=n_next.t, out=out2.t)
    other.layer(n_next.t, wr, None, ex, residual=out.t)
    assert torch.equal(out2.t, other.out)
    assert all(o.ok() for o in (n, out, n_next, ref, out2))


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces do not disturb each
    other; the bits are those of one stream."""
    T, H = 3000, 1280
    g = Gen(3)
    sets = []
    for _ in range(2):
        norm = M.make_norm(T, H, "bf16", eps=EPS)
        t = dict(norm=norm, x=g(T, H, dtype=torch.bfloat16), w=g(H, mean=1.0, dtype=torch.bfloat16),
                 dn=g(T, H, dtype=torch.bfloat16), dx=torch.empty(T, H, dtype=torch.bfloat16, device=DEV),
                 dw=torch.empty(H, device=DEV), n=torch.empty(T, H, dtype=torch.bfloat16, device=DEV))
        t["ws"], t["nb"] = workspace(norm)
        sets.append(t)

    def call(t, stream):
        M.moe_norm_in(t["norm"], t["x"], t["w"], t["n"], stream=stream)
        M.moe_norm_in_backward(t["norm"], t["dn"], t["x"], t["w"], t["n"], t["dx"], t["dw"], t["ws"],
                               t["nb"], stream=stream)

    want = []
    for t in sets:
        call(t, None)
        want.append({n: t[n].clone() for n in ("n", "dx", "dw")})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for t, s in zip(sets, streams):
            call(t, s)
    torch.cuda.synchronize()
    for t, w in zip(sets, want):
        for n in w:
            assert torch.equal(t[n], w[n]), n
