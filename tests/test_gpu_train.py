"""Training of the routed experts on the GPU against its 64-bit definitions
(tests/train_ref.py), at the sizes, routes and special values where it can go
wrong."""
import pytest
import torch

import sparse_moe_routed_amd as M
from tests import train_ref as R

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 256


class Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def __call__(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std).to(dtype)

    def integers(self, *shape, lo=-3, hi=4, dtype=torch.float32):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV).to(dtype)


class Out:
    """An output tensor with sentinels behind it, filled with `fill`."""

    def __init__(self, *shape, dtype, fill=77):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + GUARD,), 99, dtype=dtype, device=DEV)
        self.t = self.buf[:n].view(*shape)
        self.t.fill_(fill)

    def ok(self):
        return bool((self.buf[self.t.numel():] == 99).all())


class Routes:
    """Permutation arrays for T tokens of k pairs each: random, or given the
    experts of every pair; `drop` of the pairs have no row."""

    def __init__(self, T, E, k, seed=0, drop=0.0, experts=None):
        g = torch.Generator().manual_seed(seed)
        if experts is None:
            experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]) if T else \
                torch.zeros(0, k, dtype=torch.int64)
        self.ids = experts.reshape(T, k)
        ex = self.ids.reshape(-1).clone()
        ex[torch.rand(T * k, generator=g) < drop] = E
        order = torch.argsort(ex, stable=True)
        offsets = torch.zeros(E + 1, dtype=torch.int64)
        offsets[1:] = torch.cumsum(torch.bincount(ex, minlength=E + 1)[:E], 0)
        self.rows = int(offsets[E])
        pair = torch.full((T * k,), -1, dtype=torch.int64)
        pair[:self.rows] = order[:self.rows]
        dev = lambda t: t.to(torch.int32).to(DEV).contiguous()
        self.topk_ids, self.offsets, self.pair = dev(self.ids), dev(offsets), dev(pair)
        self.perm = M.make_perm(None, self.offsets, self.pair, None, None, None)


def workspace(shape):
    n = M.moe_train_workspace_size(shape)
    # NaN in every type: nothing may be taken from it that the call did not write
    return torch.full((max(n, 1) + GUARD,), 0xFF, dtype=torch.uint8, device=DEV), n


class Case:
    """Inputs, outputs and one call each of the gated product and its gradient."""

    def __init__(self, T, H, E, I, k, act="bf16", kept="act", x8=False, drop=0.0, seed=0, experts=None, ints=False):
        dt = DT[act]
        g = Gen(1000 * seed + T + H + I)
        P = T * k
        self.dims, self.dt, self.kept, self.act = (T, H, E, I, k, P), dt, kept, act
        rnd = (lambda *s, std=1.0: g.integers(*s, dtype=dt)) if ints else (lambda *s, std=1.0: g(*s, std=std, dtype=dt))
        self.rt = Routes(T, E, k, seed, drop, experts)
        self.x = rnd(T, H)
        self.w = [rnd(E, I, H, std=0.5 / H ** 0.5), rnd(E, I, H, std=0.5 / H ** 0.5), rnd(E, H, I, std=0.5 / I ** 0.5)]
        self.dy = rnd(P, H)
        self.g, self.u = rnd(P, I, std=2.0), rnd(P, I, std=2.0)
        self.shape = M.make_shape(T, H, E, I, k, act)
        self.ex = M.make_experts(*self.w)
        self.ws, self.nb = workspace(self.shape)
        self.h = Out(P, I, dtype=dt)
        if kept == "8bit":
            self.g_out, self.u_out = Out(P, I, dtype=torch.int8), Out(P, I, dtype=torch.int8)
            self.gs, self.us = Out(P, I // 32, dtype=torch.uint8), Out(P, I // 32, dtype=torch.uint8)
        else:
            self.g_out, self.u_out, self.gs, self.us = Out(P, I, dtype=dt), Out(P, I, dtype=dt), None, None
        t = lambda o: None if o is None else o.t
        self.saved = M.make_saved(self.g_out.t, self.u_out.t, t(self.gs), t(self.us))
        self.drows = Out(P, H, dtype=dt)
        self.dw = [Out(E, I, H, dtype=dt), Out(E, I, H, dtype=dt), Out(E, H, I, dtype=dt)]
        self.dex = M.make_experts(*(o.t for o in self.dw))
        self.x_in, self.x_scale = self.x, None
        if x8:
            self.x_scale = R.scales8(self.x.double())
            self.x_in = R.codes8(self.x.double(), self.x_scale)
            self.x = R.values8(self.x_in, self.x_scale)

    def outs(self):
        return [o for o in (self.h, self.g_out, self.u_out, self.gs, self.us, self.drows, *self.dw) if o is not None]

    def ok(self):
        return all(o.ok() for o in self.outs()) and bool((self.ws[self.nb:] == 0xFF).all())

    # -- the gated product --
    def save(self, stream=None):
        M.moe_ffn_gate_up_save(self.shape, self.x_in, self.ex, self.rt.perm, self.saved, self.h.t, self.ws, self.nb,
                               stream=stream)

    def check_save(self, what):
        T, H, E, I, k, P = self.dims
        want = R.gate_up(self.x, self.w[0], self.w[1], self.rt.offsets, self.rt.pair, k, self.dt)
        n = self.rt.rows
        got = {"h": self.h.t}
        if self.kept == "act":
            got.update(g=self.g_out.t, u=self.u_out.t)
            want.update({m: R._round(*want[m], self.dt) for m in ("g", "u")})
        else:
            for m, o, s in (("g", self.g_out, self.gs), ("u", self.u_out, self.us)):
                v, err = want[m][0][:n], want[m][1][:n]
                b = s.t[:n].long()
                top = lambda x: x.reshape(n, I // 32, 32).amax(2)
                hi, lo = top(v.abs() + err), top((v.abs() - err).clamp(min=0))
                assert bool((127 * R.pow2(b - 127) >= lo).all()), (what, m, "scale too small")
                assert bool(((127 * R.pow2(b - 128) < hi) | (b == 1)).all()), (what, m, "scale too large")
                step = R.pow2(b - 127).repeat_interleave(32, 1)
                back = R.values8(o.t[:n], s.t[:n])
                assert bool(((back - v).abs() <= step / 2 + err).all()), (what, m)
        R.check(got, want, what)
        # rows that no pair has are left alone
        for o in (self.h, self.g_out, self.u_out, self.gs, self.us):
            if o is not None:
                assert bool((o.t[n:] == 77).all()), what
        assert self.ok(), what

    # -- its gradient --
    def fill_saved(self):
        """Puts given g and u where the gated product would leave them."""
        if self.kept == "8bit":
            for v, o, s in ((self.g, self.g_out, self.gs), (self.u, self.u_out, self.us)):
                s.t.copy_(R.scales8(v.double()))
                o.t.copy_(R.codes8(v.double(), s.t))
            self.g, self.u = R.values8(self.g_out.t, self.gs.t), R.values8(self.u_out.t, self.us.t)
        else:
            self.g_out.t.copy_(self.g)
            self.u_out.t.copy_(self.u)

    def backward(self, drows=True, dexperts=True, stream=None):
        M.moe_ffn_backward(self.shape, self.dy, self.x_in if dexperts else None, self.x_scale if dexperts else None,
                           self.saved, self.ex, self.rt.perm, self.drows.t if drows else None,
                           self.dex if dexperts else None, self.ws, self.nb, stream=stream)

    def grads(self):
        return dict(drows=self.drows.t, dgate=self.dw[0].t, dup=self.dw[1].t, ddown=self.dw[2].t)

    def check_backward(self, what):
        want = R.backward(self.dy, self.x, self.g, self.u, *self.w, self.rt.offsets, self.rt.pair, self.dims[4], self.dt)
        R.check(self.grads(), want, what)
        assert bool((self.drows.t[self.rt.rows:] == 77).all()), what
        assert self.ok(), what


SIZES = [
    # T, H, E, I, k
    (1, 128, 1, 32, 1),          # one token through a block of its own
    (1, 128, 4, 32, 3),
    (3, 128, 1024, 32, 7),       # the most experts, most of them without a row
    (16, 256, 16, 64, 2),
    (31, 384, 5, 96, 2),         # I past a tile's half, ragged rows
    (33, 128, 1, 160, 1),        # one row more than a short tile
    (130, 256, 1, 128, 1),       # two rows more than a long tile
    (257, 128, 3, 224, 3),       # every token to every expert
    (100, 640, 7, 352, 2),
    (700, 128, 2, 32, 1),
]
FORMS = [("bf16", "act", False), ("bf16", "8bit", True), ("f32", "act", False), ("f32", "8bit", False)]


@pytest.mark.parametrize("act,kept,x8", FORMS)
@pytest.mark.parametrize("T,H,E,I,k", SIZES)
def test_gate_up_save(T, H, E, I, k, act, kept, x8):
    c = Case(T, H, E, I, k, act, kept)
    c.save()
    c.check_save(f"save {T} {H} {E} {I} {k} {act} {kept}")


@pytest.mark.parametrize("act,kept,x8", FORMS)
@pytest.mark.parametrize("T,H,E,I,k", SIZES)
def test_ffn_backward(T, H, E, I, k, act, kept, x8):
    c = Case(T, H, E, I, k, act, kept, x8)
    c.fill_saved()
    c.backward()
    c.check_backward(f"backward {T} {H} {E} {I} {k} {act} {kept}")


@pytest.mark.parametrize("drop", [0.3, 1.0])
@pytest.mark.parametrize("T,E,k", [(60, 6, 2), (400, 3, 2)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_dropped_pairs(T, E, k, act, drop):
    """Rows behind the last expert's are neither read nor written; an expert
    without rows has zero gradients."""
    c = Case(T, 128, E, 64, k, act, "8bit", drop=drop, seed=5)
    n = c.rt.rows
    c.dy[n:] = float("nan")
    c.save()
    c.check_save(f"dropped {drop}")
    c.fill_saved()
    c.gs.t[n:] = 255
    c.backward()
    c.check_backward(f"dropped {drop}")
    if drop == 1.0:
        assert n == 0 and all(bool((o.t == 0).all()) for o in c.dw)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_all_rows_on_one_expert(act):
    T, E = 300, 40
    c = Case(T, 256, E, 64, 1, act, experts=torch.full((T, 1), 17), seed=6)
    c.save()
    c.check_save("one expert")
    c.fill_saved()
    c.backward()
    c.check_backward("one expert")
    assert all(bool((o.t[:17] == 0).all()) and bool((o.t[18:] == 0).all()) for o in c.dw)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H,I", [(2560, 32), (1152, 160)])
def test_strips_of_many_experts(H, I, act):
    """Enough tiles of weight gradients that a workgroup takes several side by
    side: experts without rows, with one stage of rows, two, and many."""
    T, E = 1500, 1024
    g = torch.Generator().manual_seed(13)
    experts = torch.randint(0, E, (T, 1), generator=g)
    for e, n in ((3, 300), (5, 100), (1023, 70), (700, 64), (701, 65), (702, 128), (703, 129)):
        experts[torch.randperm(T, generator=g)[:n]] = e
    c = Case(T, H, E, I, 1, act, experts=experts, seed=13)
    c.fill_saved()
    c.backward()
    c.check_backward(f"strips {H} {I} {act}")
    first = {n: v.clone() for n, v in c.grads().items()}
    for _ in range(3):
        c.backward()
        assert all(torch.equal(v, first[n]) for n, v in c.grads().items())


# Sizes whose products are cut differently: tiles of 32, 128 and 256 rows, found by
# the workgroups (up to 64 experts) or listed, sums whole or in parts, weights
# read once or often; the last number of columns and rows inside a tile.
CUTS = [
    ("bf16", "act", 4096, 512, 1, 1056, 1), ("bf16", "8bit", 3000, 256, 70, 160, 10),
    ("bf16", "8bit", 6000, 640, 2, 2080, 2), ("bf16", "act", 2500, 384, 2, 416, 1),
    ("bf16", "8bit", 100, 2560, 8, 640, 8), ("bf16", "act", 900, 640, 70, 640, 8),
    ("bf16", "8bit", 64, 2560, 1, 640, 1), ("bf16", "8bit", 140, 2560, 66, 32, 1),
    ("bf16", "act", 4612, 2560, 1, 96, 1), ("f32", "act", 6000, 640, 2, 2080, 2),
    ("f32", "8bit", 3000, 256, 70, 160, 10), ("f32", "8bit", 4100, 1280, 1, 2080, 1),
    ("f32", "act", 2500, 384, 2, 416, 1), ("f32", "8bit", 130, 1280, 70, 320, 10),
    ("f32", "act", 900, 640, 70, 640, 8), ("f32", "8bit", 200, 2560, 1, 96, 1),
    # the last tiles' sums cut
    ("bf16", "act", 7000, 768, 1, 1600, 1), ("bf16", "8bit", 8000, 1152, 1, 1280, 1),
    ("bf16", "8bit", 6500, 1280, 1, 2592, 1), ("bf16", "act", 6100, 1280, 5, 1056, 2),
    ("f32", "act", 7000, 768, 1, 1600, 1), ("f32", "8bit", 8000, 1024, 1, 1056, 1)]


@pytest.mark.parametrize("act,kept,T,H,E,I,k", CUTS)
def test_every_cut(act, kept, T, H, E, I, k):
    c = Case(T, H, E, I, k, act, kept, drop=0.1, seed=17)
    c.save()
    c.check_save(f"cut {T} {H} {E} {I} {k} {act} {kept}")
    c = Case(T, H, E, I, k, act, kept, kept == "8bit", drop=0.1, seed=18)
    c.fill_saved()
    c.backward()
    c.check_backward(f"cut {T} {H} {E} {I} {k} {act} {kept}")
    first = {n: v.clone() for n, v in c.grads().items()}
    c.backward()
    assert all(torch.equal(v, first[n]) for n, v in c.grads().items())


@pytest.mark.parametrize("kept", ["act", "8bit"])
@pytest.mark.parametrize("T,E,k", [(50, 9, 2), (260, 2, 2)])
def test_small_integers_are_exact(T, E, k, kept):
    """Products of small integers are exact in float32, so g, u and the codes
    have exactly one right answer."""
    c = Case(T, 128, E, 96, k, "bf16", kept, ints=True, seed=7)
    c.save()
    n = c.rt.rows
    tok = c.rt.pair[:n].long() // k
    ex = torch.repeat_interleave(torch.arange(E, device=DEV), c.rt.offsets.diff().long())
    for w, o, s in ((c.w[0], c.g_out, c.gs), (c.w[1], c.u_out, c.us)):
        v = torch.stack([w[int(e)].double() @ c.x[int(t)].double() for e, t in zip(ex, tok)])
        if kept == "act":
            assert torch.equal(o.t[:n], v.to(c.dt))
        else:
            assert torch.equal(s.t[:n], R.scales8(v))
            assert torch.equal(o.t[:n], R.codes8(v, s.t[:n]))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (500, 4, 2)])
def test_special_values_stay_with_their_rows(T, E, k, act):
    """A NaN or infinity in one token's x or one row's dy reaches that row, the
    gradients of its expert, and nothing else."""
    base = Case(T, 128, E, 64, k, act, seed=8)
    base.fill_saved()
    base.save()
    h0 = base.h.t.clone()
    base.fill_saved()
    base.backward()
    clean = {n: v.clone() for n, v in base.grads().items()}
    for bad in (float("nan"), float("inf")):
        c = Case(T, 128, E, 64, k, act, seed=8)
        token, row = 5, c.rt.rows // 2
        c.x[token, 9] = bad
        c.save()
        tok = c.rt.pair.long() // k
        assert torch.equal(c.h.t[tok != token], h0[tok != token])
        assert not bool(torch.isfinite(c.h.t[tok == token]).any())
        c = Case(T, 128, E, 64, k, act, seed=8)
        c.fill_saved()
        c.x[token, 9] = bad
        c.dy[row, 3] = bad
        c.backward()
        got = c.grads()
        others = torch.ones(T * k, dtype=torch.bool, device=DEV)
        others[row] = False
        assert torch.equal(got["drows"][others], clean["drows"][others])
        assert not bool(torch.isfinite(got["drows"][row]).any())
        ex = torch.repeat_interleave(torch.arange(E, device=DEV), c.rt.offsets.diff().long())
        hit = set(ex[tok == token].tolist()) | {int(ex[row])}
        for e in range(E):
            for n in ("dgate", "dup", "ddown"):
                if e not in hit:
                    assert torch.equal(got[n][e], clean[n][e]), (n, e)
        # x's bad column is that column of the expert's gradients, no more
        e = int(ex[tok == token][0])
        if e != int(ex[row]):
            cols = torch.arange(128, device=DEV) != 9
            assert torch.equal(got["dgate"][e][:, cols], clean["dgate"][e][:, cols])
            assert not bool(torch.isfinite(got["dgate"][e][:, 9]).any())
            assert torch.equal(got["ddown"][e], clean["ddown"][e])


def test_extreme_gates():
    """g far outside exp's range: silu and its slope saturate, no NaN."""
    for act in ("bf16", "f32"):
        c = Case(20, 128, 3, 32, 1, act, seed=9)
        c.g[:, ::4] = 300.0
        c.g[:, 1::4] = -300.0
        c.g[:, 2::4] = -88.5
        c.fill_saved()
        c.backward()
        assert all(bool(torch.isfinite(v).all()) for v in c.grads().values())
        c.check_backward(f"extreme gates {act}")


def test_a_gradient_that_is_not_wanted_is_not_written():
    for act in ("bf16", "f32"):
        c = Case(90, 256, 5, 96, 2, act, seed=10)
        c.fill_saved()
        c.backward()
        want = {n: v.clone() for n, v in c.grads().items()}
        for kw in (dict(drows=False), dict(dexperts=False)):
            for o in (c.drows, *c.dw):
                o.t.fill_(77)
            c.backward(**kw)
            for n, v in c.grads().items():
                skipped = n == "drows" if "drows" in kw else n != "drows"
                assert bool((v == 77).all()) if skipped else torch.equal(v, want[n]), (kw, n)


def test_empty_batch_clears_the_weights_gradients():
    for act in ("bf16", "f32"):
        H, E, I = 256, 5, 96
        dw = [Out(E, I, H, dtype=DT[act]), Out(E, I, H, dtype=DT[act]), Out(E, H, I, dtype=DT[act])]
        s = M.make_shape(0, H, E, I, 2, act)
        M.moe_ffn_backward(s, None, None, None, None, None, None, None, M.make_experts(*(o.t for o in dw)), None, 0)
        assert all(bool((o.t == 0).all()) and o.ok() for o in dw)
        dwr, db = Out(E, H, dtype=torch.float32), Out(E, dtype=torch.float32)
        M.moe_router_backward(s, None, None, None, None, None, None, None, None, dwr.t, db.t, None, 0)
        assert bool((dwr.t == 0).all()) and bool((db.t == 0).all()) and dwr.ok() and db.ok()


@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (600, 3, 2)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_indices_out_of_range_are_memory_safe(T, E, k, act):
    """Offsets and pairs that no permutation has: the call ends and writes
    inside its outputs."""
    g = torch.Generator().manual_seed(11)
    c = Case(T, 128, E, 64, k, act, "8bit", seed=11)
    c.fill_saved()
    big = 2 ** 31 - 1
    for kind in range(3):
        c.rt.offsets.copy_(torch.tensor([[big] * (E + 1), [-big] + [big] * E,
                                         torch.randint(-5, 2 * T * k, (E + 1,), generator=g).tolist()][kind],
                                        dtype=torch.int32))
        c.rt.pair.copy_(torch.randint(-big, big, (T * k,), generator=g, dtype=torch.int32))
        c.save()
        c.backward()
        torch.cuda.synchronize()
        assert c.ok(), kind


# ---- 8-bit checkpoints ----


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2560), (7, 96), (3, 8192), (1001, 160), (40000, 64)])
def test_checkpoint(rows, cols, act):
    dt, g = DT[act], Gen(rows + cols)
    v = (g(rows, cols) * torch.exp(3 * g(1, cols))).to(dt)
    codes, scales = Out(rows, cols, dtype=torch.int8), Out(rows, cols // 32, dtype=torch.uint8)
    M.moe_save8(act, rows, cols, v, codes.t, scales.t)
    s = R.scales8(v.double())
    assert torch.equal(scales.t, s) and torch.equal(codes.t, R.codes8(v.double(), s))
    back = Out(rows, cols, dtype=dt)
    M.moe_restore8(act, rows, cols, codes.t, scales.t, back.t)
    assert torch.equal(back.t.double(), R.values8(codes.t, s))
    assert codes.ok() and scales.ok() and back.ok()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_checkpoint_special_values(act):
    """Zeros, subnormals, the borders of the scales, the largest numbers, ties,
    infinities and NaN."""
    dt = DT[act]
    inf, nan = float("inf"), float("nan")
    tops = [0.0, 2.0 ** -133, 2.0 ** -126, 127 * 2.0 ** -126, 127.5 * 2.0 ** -126, 1.0, 1.984375, 1.9921875, 2.0,
            127.0, 127.5, 128.0, 3.38e38, inf, -inf, nan, -0.0, 1e-30]
    v = torch.zeros(len(tops), 32, dtype=dt, device=DEV)
    for i, t in enumerate(tops):
        scale = 1.0 if t != t or abs(t) == inf or t == 0 else abs(t)
        v[i] = (torch.linspace(-1, 1, 32, device=DEV) * scale * 0.99).to(dt)
        v[i, 13] = t
        v[i, 5] = 0.5 * 2.0 ** -126                              # half a code of the smallest scale
        if t == 0:
            v[i] = t
    if act == "f32":
        v[5, 20] = 1.0000001
    codes = torch.full((len(tops), 32), 77, dtype=torch.int8, device=DEV)
    scales = torch.zeros(len(tops), 1, dtype=torch.uint8, device=DEV)
    M.moe_save8(act, len(tops), 32, v, codes, scales)
    s = R.scales8(v.double())
    assert torch.equal(scales, s), (scales.flatten(), s.flatten())
    assert torch.equal(codes, R.codes8(v.double(), s))
    back = torch.empty_like(v)
    M.moe_restore8(act, len(tops), 32, codes, scales, back)
    want = R.values8(codes, s)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.double().nan_to_num(), want.nan_to_num())
    assert bool(torch.isnan(back[13:16]).all()) and not bool(torch.isnan(back[:13]).any())


def test_every_code_and_scale_reads_back():
    for act in ("bf16", "f32"):
        codes = torch.arange(-128, 128, device=DEV).to(torch.int8).repeat(256, 1)
        scales = torch.arange(256, device=DEV).to(torch.uint8)[:, None].repeat(1, 8)
        v = torch.empty(256, 256, dtype=DT[act], device=DEV)
        M.moe_restore8(act, 256, 256, codes, scales, v)
        want = R.values8(codes, scales)
        want = want.to(torch.float32).to(DT[act])               # 2^127 * 127 is past float32
        assert torch.equal(torch.isnan(v), torch.isnan(want)) and torch.equal(v.nan_to_num(7), want.nan_to_num(7))


# ---- the router's product ----


class RouterCase:
    def __init__(self, T, H, E, k, act, dx_in=True, seed=0, experts=None):
        g, dt = Gen(seed + T + H + E), DT[act]
        self.dims, self.dt = (T, H, E, k), dt
        self.rt = Routes(T, E, k, seed, experts=experts)
        self.x, self.wr = g(T, H, dtype=dt), g(E, H, std=0.1, dtype=dt)
        self.w, self.dw = torch.softmax(g(T, k), dim=1), g(T, k)
        self.dx_in = g(T, H, dtype=dt) if dx_in else None
        self.shape = M.make_shape(T, H, E, 32, k, act)
        self.ws, self.nb = workspace(self.shape)
        self.dx, self.dwr = Out(T, H, dtype=dt), Out(E, H, dtype=torch.float32)
        self.db = Out(E, dtype=torch.float32)

    def call(self, dx=True, dwr=True, db=True, stream=None):
        M.moe_router_backward(self.shape, self.rt.topk_ids, self.w, self.dw, self.x if dwr else None,
                              self.wr if dx else None, self.rt.perm if dwr or db else None,
                              self.dx_in if dx else None, self.dx.t if dx else None, self.dwr.t if dwr else None,
                              self.db.t if db else None, self.ws, self.nb, stream=stream)

    def got(self):
        return dict(dx=self.dx.t, dw_router=self.dwr.t, dbias=self.db.t)

    def check(self, what):
        R.check(self.got(), R.router(self.rt.topk_ids, self.w, self.dw, self.x, self.wr, self.dx_in, self.dt), what)
        assert self.dx.ok() and self.dwr.ok() and self.db.ok() and bool((self.ws[self.nb:] == 0xFF).all())


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E,k,dx_in", [
    (1, 128, 2, 2, False), (1, 2560, 512, 10, True), (17, 384, 9, 3, True), (333, 384, 60, 3, False),
    (300, 128, 400, 300, True), (5, 4096, 1024, 1024, True), (2000, 256, 3, 2, True), (1500, 1280, 128, 8, False)])
def test_router_backward(T, H, E, k, dx_in, act):
    c = RouterCase(T, H, E, k, act, dx_in)
    c.call()
    c.check(f"router {T} {H} {E} {k} {act}")
    # against the logits' gradient that moe_route_backward gives
    dl = torch.empty(T, E, device=DEV)
    M.moe_route_backward(c.shape, c.rt.topk_ids, c.w, c.dw, dl)
    want = dl.double().sum(0)
    bound = (T + 4) * R.E * dl.double().abs().sum(0) * 2 + 1e-30
    # both round each dl: by the k terms of its sum at most
    bound = bound + (k + 8) * R.E * (c.w.double() * (c.dw.double().abs() + (c.w * c.dw).double().abs().sum(1, keepdim=True))).sum() * 2
    assert bool(((c.db.t.double() - want).abs() <= bound).all())


def test_router_parts_that_are_not_wanted():
    c = RouterCase(200, 256, 12, 4, "bf16", seed=3)
    c.call()
    want = {n: v.clone() for n, v in c.got().items()}
    for skip in ("dx", "dwr", "db"):
        for o in (c.dx, c.dwr, c.db):
            o.t.fill_(77)
        c.call(**{skip: False})
        name = dict(dx="dx", dwr="dw_router", db="dbias")[skip]
        for n, v in c.got().items():
            assert bool((v == 77).all()) if n == name else torch.equal(v, want[n]), (skip, n)


def test_router_ids_out_of_range_add_nothing():
    c = RouterCase(40, 256, 8, 2, "f32", dx_in=False)
    c.rt.topk_ids[3, 1], c.rt.topk_ids[7, 0] = 8, -1
    c.call(dwr=False, db=False)
    ids = c.rt.topk_ids.clone()
    w0 = torch.zeros(10, 256, device=DEV)
    w0[:8] = c.wr
    ids[3, 1], ids[7, 0] = 8, 9                                  # rows of zeros
    want = R.router(ids, c.w, c.dw, c.x, w0, None, torch.float32)
    R.check({"dx": c.dx.t}, want, "ids out of range")
    assert c.dx.ok()


# ---- together ----


class Layer:
    """A layer of MoELayerBuffers with all that training it takes."""

    def __init__(self, T=50, H=256, E=12, I=96, k=3, act="f32", kept="act", seed=1):
        g, dt = Gen(seed), DT[act]
        self.dims, self.act, self.kept = (T, H, E, I, k), act, kept
        self.buf = M.MoELayerBuffers(T, H, E, I, k, act, device=DEV)
        self.x, self.wr = g(T, H, dtype=dt), g(E, H, std=0.05, dtype=dt)
        self.bias = g(E, std=0.1)
        self.w = [g(E, *s, std=0.05, dtype=dt) for s in ((I, H), (I, H), (H, I))]
        self.ex = M.make_experts(*self.w)
        self.dout = g(T, H, dtype=dt)
        self.dx = torch.empty_like(self.x)
        self.dwr, self.db = torch.empty(E, H, device=DEV), torch.empty(E, device=DEV)
        self.dw = [torch.empty_like(w) for w in self.w]
        self.dex = M.make_experts(*self.dw)

    def step(self, stream=None):
        self.buf.layer_save(self.x, self.wr, self.bias, self.ex, residual=self.x, kept=self.kept, stream=stream)
        self.buf.layer_backward(self.dout, self.x, self.wr, self.ex, self.dx, self.dwr, self.db, self.dex,
                                dx_in=self.dout, stream=stream)

    def outputs(self):
        return dict(out=self.buf.out, h=self.buf.h, g=self.buf.g, u=self.buf.u, dx=self.dx, dwr=self.dwr, db=self.db,
                    dgate=self.dw[0], dup=self.dw[1], ddown=self.dw[2])


@pytest.mark.parametrize("T,H,E,I,k", [(50, 256, 12, 96, 3), (300, 128, 4, 64, 2), (7, 384, 64, 32, 5)])
def test_layer_gradients_match_autograd(T, H, E, I, k):
    """layer_save and layer_backward against torch's differentiation of the
    layer in float64 for the same routes.  Sums of at most H = 384 terms
    (rounding 2 (H + 2) 2^-24 = 5e-5 of the magnitudes at worst, the root of
    that many at random), five products in a row, none cancelling by more than
    ten in the norm of a whole output: 2e-4 relative in norm."""
    b = Layer(T, H, E, I, k)
    b.step()
    D = dict(x=b.x, wr=b.wr, bias=b.bias, w0=b.w[0], w1=b.w[1], w2=b.w[2])
    D = {n: v.double().requires_grad_() for n, v in D.items()}
    ids = b.buf.topk_ids.long()
    w = torch.softmax((D["x"] @ D["wr"].t() + D["bias"]).gather(1, ids), 1)
    out = D["x"]
    for j in range(k):
        e = ids[:, j]
        g = (D["w0"][e] * D["x"][:, None, :]).sum(2)
        u = (D["w1"][e] * D["x"][:, None, :]).sum(2)
        out = out + w[:, j, None] * (D["w2"][e] * (g * torch.sigmoid(g) * u)[:, None, :]).sum(2)
    (out * b.dout.double()).sum().backward()
    rel = lambda a, r: float((a.double() - r).norm() / r.norm())
    for name, got, want in (("out", b.buf.out, out.detach()), ("dx", b.dx, D["x"].grad), ("dwr", b.dwr, D["wr"].grad),
                            ("db", b.db, D["bias"].grad), ("dgate", b.dw[0], D["w0"].grad),
                            ("dup", b.dw[1], D["w1"].grad), ("ddown", b.dw[2], D["w2"].grad)):
        assert rel(got, want) <= 2e-4, (name, rel(got, want))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_layer_save_is_the_layer(act):
    """The training forward gives the layer's output, within the rounding of h:
    h to the act type (u), y to the act type (u), out to the act type (u) and
    sums of 256 terms; the magnitudes added are those of the absolute values."""
    b = Layer(act=act)
    b.buf.layer_save(b.x, b.wr, b.bias, b.ex, residual=b.x)
    out, ids = b.buf.out.clone(), b.buf.topk_ids.clone()
    T, H, E, I, k = b.dims
    other = M.MoELayerBuffers(T, H, E, I, k, act, device=DEV)
    other.layer(b.x, b.wr, b.bias, b.ex, residual=b.x)
    assert torch.equal(ids, other.topk_ids)
    u = R.u_of(DT[act])
    h = R.gate_up(b.x, b.w[0], b.w[1], b.buf.offsets, b.buf.sorted_pair, k, DT[act])["h"]
    row = b.buf.pair_row.reshape(T, k).long()
    mag, err = b.x.double().abs(), 0
    for j in range(k):
        wd = b.w[2][ids[:, j].long()].double().abs()
        y = (wd * h[0][row[:, j]].abs()[:, None, :]).sum(2)
        ey = (wd * h[1][row[:, j]][:, None, :]).sum(2) + 2 * (I + 2) * R.E * y
        w = b.buf.topk_w[:, j, None].double()
        err = err + w * (ey + y * u)
        mag = mag + w * y
    bound = 2 * (err + (k + 2) * R.E * mag + mag * u)              # either side
    assert bool(((out.double() - other.out.double()).abs() <= bound).all())


@pytest.mark.parametrize("act,kept", [("bf16", "8bit"), ("f32", "act")])
@pytest.mark.parametrize("T,E", [(50, 12), (900, 4)])
def test_step_in_a_graph_repeats(act, kept, T, E):
    """Captured once, replayed with eager work and new inputs between: every
    replay has the bits of the eager run on the same inputs."""
    b = Layer(T=T, E=E, act=act, kept=kept)
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for i in range(4):
        b.x.copy_(Gen(70 + i)(*b.x.shape, dtype=b.x.dtype))
        b.step()
        torch.cuda.synchronize()
        want = {n: v.clone() for n, v in b.outputs().items()}
        for v in b.outputs().values():
            v.fill_(7)
        b.buf.train_ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for n, v in b.outputs().items():
            assert torch.equal(v, want[n]), (i, n)


def test_two_streams_at_once():
    """Steps on two streams with their own buffers do not disturb each other,
    and the bits are those of one stream."""
    sets = [Layer(T=400, E=6, act="bf16", kept="8bit", seed=s) for s in (1, 2)]
    want = []
    for b in sets:
        b.step()
        torch.cuda.synchronize()
        want.append({n: v.clone() for n, v in b.outputs().items()})
        for v in b.outputs().values():
            v.fill_(7)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        for b, s in zip(sets, streams):
            b.step(stream=s)
    torch.cuda.synchronize()
    for b, w in zip(sets, want):
        for n, v in b.outputs().items():
            assert torch.equal(v, w[n]), n


def test_a_checkpoint_of_x_in_the_backward_pass():
    """layer_backward from x kept in 8 bits: the gradient for the values that
    the codes stand for."""
    b = Layer(T=60, act="bf16", kept="8bit")
    T, H = b.dims[:2]
    codes = torch.empty(T, H, dtype=torch.int8, device=DEV)
    scales = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV)
    M.moe_save8("bf16", T, H, b.x, codes, scales)
    b.buf.layer_save(b.x, b.wr, b.bias, b.ex, kept="8bit")
    grads = lambda: [t.clone() for t in (b.dx, b.dwr, b.db, *b.dw)]
    b.buf.layer_backward(b.dout, codes, b.wr, b.ex, b.dx, b.dwr, b.db, b.dex, x_scale=scales)
    got = grads()
    back = R.values8(codes, scales).to(torch.bfloat16)
    b.buf.layer_backward(b.dout, back, b.wr, b.ex, b.dx, b.dwr, b.db, b.dex)
    assert all(torch.equal(a, c) for a, c in zip(got, grads()))
    # and through the entry point itself
    c = [torch.empty_like(w) for w in b.dw]
    b.buf.ffn_backward(b.buf.dy, codes, b.ex, dexperts=M.make_experts(*c), x_scale=scales)
    assert all(torch.equal(a, d) for a, d in zip(c, b.dw))


def test_rows_past_32_bit_offsets():
    """x, dy and drows of 4 GiB each: rows at the end of the memory give the
    values of a batch of their own."""
    T, H, E, I = 131072, 16256, 2, 32
    g = Gen(12)
    s = M.make_shape(T, H, E, I, 1)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    n = 300
    tail = slice(T - n, T)
    x[tail], dy[tail] = g(n, H, dtype=torch.bfloat16), g(n, H, dtype=torch.bfloat16)
    x[0] = 1.0
    w = [g(E, *sh, std=0.05, dtype=torch.bfloat16) for sh in ((I, H), (I, H), (H, I))]
    # the first half of the tokens on expert 0
    i32 = dict(dtype=torch.int32, device=DEV)
    offsets, pair = torch.tensor([0, T // 2, T], **i32), torch.arange(T, **i32)
    perm = M.make_perm(None, offsets, pair, None, None, None)
    ws = torch.empty(M.moe_train_workspace_size(s), dtype=torch.uint8, device=DEV)
    h, gk, uk = (torch.empty(T, I, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    M.moe_ffn_gate_up_save(s, x, M.make_experts(*w), perm, M.make_saved(gk, uk), h, ws, ws.numel())
    drows = torch.empty_like(dy)
    dw = [torch.empty_like(t) for t in w]
    M.moe_ffn_backward(s, dy, x, None, M.make_saved(gk, uk), M.make_experts(*w), perm, drows, M.make_experts(*dw), ws,
                       ws.numel())
    small = torch.tensor([0, 0, n], **i32)
    want = R.gate_up(x[tail], w[0], w[1], small, pair[:n], 1, torch.bfloat16)
    R.check({"h": h[tail]}, {"h": want["h"]}, "h")
    want = R.backward(dy[tail], x[tail], gk[tail], uk[tail], *w, small, pair[:n], 1, torch.bfloat16)
    R.check({"drows": drows[tail]}, {"drows": want["drows"]}, "drows")
    # the other rows of dy are zeros, so they add nothing; the sums may be longer by T / n
    for name, t, i in (("dgate", dw[0], 1), ("dup", dw[1], 1), ("ddown", dw[2], 1)):
        v, bound = want[name]
        assert bool(((t[i].double() - v[i]).abs() <= bound[i]).all()), name
    assert all(bool((t[0] == 0).all()) for t in dw)
    assert bool((drows[:T - n] == 0).all())
