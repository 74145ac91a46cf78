"""64-bit definitions of the training of the routed experts, with bounds on the
error of a float32 computation (not a test module).

Every function returns {name: (value, bound)}: the float64 value of an output
and the largest error a correct kernel can make.  The bounds count roundings:
e = 2^-24 for each float32 operation, u = eps / 2 of a type for a rounding to
it.  A product of K terms is K multiplications and K additions in an unknown
order: at most (K + 2) e times the sum of the terms' magnitudes; a matrix
instruction may cut instead of round, which doubles it.  Underflow of float32 adds at
most TINY for each term."""
from __future__ import annotations

import torch

E = 2.0 ** -24
TINY = 2.0 ** -120


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


# ---- 8-bit checkpoints ----

def pow2(e):
    """2^e in float64, exactly (pow() on the GPU is off by some bits, which
    turns ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def scales8(v):
    """Scale bytes [..., n / 32] of a float64 matrix, from the definition: the
    smallest b >= 1 with 127 * 2^(b - 127) >= the largest magnitude, at most 248,
    255 where one is not finite."""
    g = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    top = g.abs().amax(dim=-1)
    b = torch.full_like(top, 248.0)
    for cand in range(247, 0, -1):
        b = torch.where(top <= 127.0 * 2.0 ** (cand - 127), torch.full_like(b, float(cand)), b)
    finite = torch.isfinite(g).all(dim=-1)
    return torch.where(finite, b, torch.full_like(b, 255.0)).to(torch.uint8)


def codes8(v, scales):
    step = pow2(scales.long() - 127).repeat_interleave(32, dim=-1)
    q = torch.round(v / step).clamp(-127, 127)
    return torch.where(scales.repeat_interleave(32, dim=-1) == 255, torch.zeros_like(q), q).to(torch.int8)


def values8(codes, scales):
    """float64 values of a checkpoint."""
    step = pow2(scales.long() - 127)
    step = torch.where(scales == 255, torch.full_like(step, float("nan")), step)
    return codes.double() * step.repeat_interleave(32, dim=-1)


# ---- the two products ----

def _prod(a, ea, b):
    """(a @ b, error) of float32 products of a known to ea with exact b."""
    K = a.shape[1]
    v, mag = a @ b, a.abs() @ b.abs()
    return v, 2 * (K + 2) * E * mag + ea @ b.abs() + K * TINY


def _round(v, e, dtype):
    return v, e + (v.abs() + e) * u_of(dtype) + TINY


def _sigmoid(g):
    """sigmoid and its relative error in float32: exp of a rounded product
    (|g| e of its value), then exp, addition and division, each a few e."""
    return 1 / (1 + torch.exp(-g)), (12 + 2 * g.abs()) * E


def rows_of(offsets, sorted_pair, k, e):
    a, b = int(offsets[e]), int(offsets[e + 1])
    return a, b, sorted_pair[a:b].long() // k


def gate_up(x, wg, wu, offsets, sorted_pair, k, dtype):
    """g, u, h [P][I]; rows that no pair has are NaN."""
    Ex, I, P = wg.shape[0], wg.shape[1], len(sorted_pair)
    out = {n: torch.full((2, P, I), float("nan"), dtype=torch.float64, device=x.device)
           for n in ("g", "u", "h")}
    for e in range(Ex):
        a, b, t = rows_of(offsets, sorted_pair, k, e)
        if a == b:
            continue
        xe = x[t].double()
        z = torch.zeros_like(xe)
        g, eg = _prod(xe, z, wg[e].double().t())
        u, eu = _prod(xe, z, wu[e].double().t())
        s, rs = _sigmoid(g)
        # |d silu| <= 1.1 times the error of g
        silu, es = g * s, 1.1 * eg + (g * s).abs() * (rs + 2 * E)
        h = silu * u
        eh = (es * u.abs() + silu.abs() * eu + es * eu) + h.abs() * 2 * E
        for n, (v, err) in dict(g=(g, eg), u=(u, eu), h=_round(h, eh, dtype)).items():
            out[n][0, a:b], out[n][1, a:b] = v, err
    return {n: (v[0], v[1]) for n, v in out.items()}


def backward(dy, x, g, u, wg, wu, wd, offsets, sorted_pair, k, dtype):
    """drows [P][H] (NaN where no pair has the row) and the weights' gradients.
    dy, x, g, u: the values the call was given (checkpoints read back)."""
    Ex, I, H = wg.shape
    P = len(sorted_pair)
    new = lambda *s: torch.zeros((2, *s), dtype=torch.float64, device=dy.device)
    drows, dgate, dup, ddown = new(P, H).fill_(float("nan")), new(Ex, I, H), new(Ex, I, H), new(Ex, H, I)
    for e in range(Ex):
        a, b, t = rows_of(offsets, sorted_pair, k, e)
        if a == b:
            continue
        ge, ue, dye, xe = g[a:b].double(), u[a:b].double(), dy[a:b].double(), x[t].double()
        dh, edh = _prod(dye, torch.zeros_like(dye), wd[e].double())
        s, rs = _sigmoid(ge)
        h = ge * s * ue
        du = dh * ge * s
        q = torch.exp(-ge)
        slope = torch.where(ge < -700, torch.zeros_like(ge), (1 + q + ge * q) * s * s)
        dg = dh * ue * slope
        # s (1 + g (1 - s)): each factor to a few e of 1 + |g|
        eslope = s * (1 + ge.abs()) * (2 * rs + 8 * E)
        h, eh = _round(h, h.abs() * (rs + 3 * E), dtype)
        du, edu = _round(du, edh * (ge * s).abs() + du.abs() * (rs + 3 * E), dtype)
        dg, edg = _round(dg, edh * (ue * slope).abs() + (dh * ue).abs() * eslope + edh * ue.abs() * eslope
                         + dg.abs() * 4 * E, dtype)
        v1, e1 = _prod(dg, edg, wg[e].double())
        v2, e2 = _prod(du, edu, wu[e].double())
        drows[0, a:b], drows[1, a:b] = _round(v1 + v2, (e1 + e2) * (1 + 4 * E) + 2 * I * E * (v1.abs() + v2.abs()), dtype)
        for out, m, em, n in ((dgate, dg, edg, xe), (dup, du, edu, xe)):
            v, err = _prod(m.t(), em.t(), n)
            out[0, e], out[1, e] = _round(v, err, dtype)
        v, err = _prod(h.t(), eh.t(), dye)
        v, err = _round(v, err, dtype)
        ddown[0, e], ddown[1, e] = v.t(), err.t()
    return {n: (v[0], v[1]) for n, v in
            dict(drows=drows, dgate=dgate, dup=dup, ddown=ddown).items()}


def router(ids, w, dw, x, w_router, dx_in, dtype):
    """dx, dw_router, dbias."""
    T, k = ids.shape
    Ex, H = w_router.shape
    w, dw = w.double(), dw.double()
    dot, mag = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    dl = w * (dw - dot)
    edl = w.abs() * (mag * (k + 2) * E + (dw.abs() + dot.abs()) * E) + dl.abs() * E
    full = lambda v: torch.zeros(T, Ex, dtype=torch.float64, device=x.device).scatter_(1, ids.long(), v)
    L, eL = full(dl), full(edl)
    d0 = 0 if dx_in is None else dx_in.double()
    v, err = _prod(L, eL, w_router.double())
    dx = v + d0
    # the sum has k + 1 terms that are not zero; _prod counts all E
    dx = _round(dx, err + (k + 2) * E * (v.abs() + (0 if dx_in is None else d0.abs())), dtype)
    dwr, edwr = _prod(L.t(), eL.t(), x.double())
    dwr = _round(dwr, edwr, torch.float32)
    db = L.sum(0)
    return dict(dx=dx, dw_router=dwr,
                dbias=(db, eL.sum(0) + (T + 2) * E * L.abs().sum(0) + TINY))


def check(got, want, what):
    """Every value within its bound; rows that the reference leaves NaN are skipped."""
    for name, (v, bound) in want.items():
        if name not in got:
            continue
        g = got[name].double()
        assert g.shape == v.shape, (what, name, g.shape, v.shape)
        on = ~torch.isnan(v)
        bad = on & ~((g - v).abs() <= bound)
        if bool(bad.any()):
            i = tuple(int(c) for c in bad.nonzero()[0])
            raise AssertionError(f"{what} {name}: {int(bad.sum())} of {int(on.sum())} out of bounds, first {i}: "
                                 f"{float(g[i])} for {float(v[i])} +- {float(bound[i])}")
