"""64-bit definition of a whole routed layer and its gradient for given routes, with
bounds on the error of a computation that keeps and rounds what layer_save and
layer_backward do (not a test module).

Every value goes on with the largest error that it can have: sums in float32
(tests/train_ref.py: at most 2 (K + 2) 2^-24 of the magnitudes' sum), half a step of
the type at each tensor in memory (h, y, out, dy, dg, du, drows, dx), half a code
where g and u are kept in 8 bits, and EW for the routes' weights.  They are the worst
case of every term, so wide where long sums of rounded values follow each other; the
steps one by one are held to their own bounds beside this."""
from __future__ import annotations

import torch

from tests.train_ref import E, TINY, u_of

EW = 1e-5        # of a route's weight, as everywhere in the GPU tests


class V:
    """A float64 value and the largest error of what stands for it."""

    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def top(self):
        return self.v.abs() + self.e

    def __add__(self, o):
        return V(self.v + o.v, self.e + o.e)

    def __mul__(self, o):
        """One rounded product."""
        v = self.v * o.v
        t = self.top() * o.top()
        return V(v, t - v.abs() + t * E + TINY)

    def round(self, dtype):
        return V(self.v, self.e + self.top() * u_of(dtype) + TINY)

    def map(self, f):
        return V(f(self.v), f(self.e))


def dot(a, b, how, terms):
    """einsum of two values, `terms` float32 products and sums each."""
    v = torch.einsum(how, a.v, b.v)
    t = torch.einsum(how, a.top(), b.top())
    exact = torch.einsum(how, a.v.abs(), b.v.abs())
    return V(v, t - exact + 2 * (terms + 2) * E * t + terms * TINY)


def total(a, dim, terms):
    return V(a.v.sum(dim), a.e.sum(dim) + 2 * (terms + 2) * E * a.top().sum(dim))


def _sigmoid(g):
    """With its relative error in float32 (tests/train_ref.py)."""
    return 1 / (1 + torch.exp(-g)), (12 + 2 * g.abs()) * E


def silu(g):
    s, rel = _sigmoid(g.v)
    v = g.v * s
    return V(v, 1.1 * g.e + v.abs() * (rel + 2 * E) + TINY)     # |silu'| <= 1.1


def slope(g):
    """silu'(g); |silu''| <= 1/2."""
    s, rel = _sigmoid(g.v)
    q = torch.exp(-g.v)
    return V((1 + q + g.v * q) * s * s, 0.5 * g.e + s * (1 + g.v.abs()) * (2 * rel + 8 * E) + TINY)


def kept(g, how, dtype):
    """g as the gradient reads it."""
    if how == "act":
        return g.round(dtype)
    # a scale is less than twice what the largest of 32 needs, so half a code is at most 1 / 127 of it
    top = g.top().reshape(g.v.shape[0], -1, 32).amax(2) / 127 + 2.0 ** -127
    return V(g.v, g.e + top.repeat_interleave(32, 1))


def layer(x, wr, bias, w, ids, residual, dout, dx_in, dtype, how, mistake=None):
    """out, dx, dwr, db, dgate, dup, ddown as V; w: gate, up, down; ids [T][k].
    `mistake` leaves a part out, to show that the bounds notice."""
    x, wr, dout, w = x.double(), wr.double(), dout.double(), [t.double() for t in w]
    T, k = ids.shape
    Ex, I, H = w[0].shape
    ids = ids.long()
    pair = ids.reshape(-1)
    token = torch.arange(T, device=x.device).repeat_interleave(k)
    logits = x @ wr.t() + bias.double()
    weight = torch.softmax(logits.gather(1, ids), 1)
    wt = V(weight, torch.full_like(weight, EW))
    if mistake == "even weights":
        wt = V(torch.full_like(weight, 1 / k), wt.e)
    rows = V(x[token])
    W = [V(t[pair]) for t in w]
    if mistake == "gate and up swapped":
        W[0], W[1] = W[1], W[0]

    g, u = (dot(rows, m, "ph,pih->pi", H) for m in W[:2])
    h = (silu(g) * u).round(dtype)
    y = dot(h, W[2], "pi,phi->ph", I).round(dtype)
    by_token = lambda v: v.map(lambda t: t.reshape(T, k, -1))
    wp = wt.map(lambda t: t.reshape(T, k, 1))
    out = total(by_token(y) * wp, 1, k + 1) + V(residual.double())
    out = V(out.v, out.e + (k + 3) * E * out.top()).round(dtype)

    dy = V(dout[token]) * wt.map(lambda t: t.reshape(-1, 1))
    dy = dy.round(dtype)
    dw = dot(V(dout[token]), y, "ph,ph->p", H).map(lambda t: t.reshape(T, k))
    dh = dot(dy, W[2], "ph,phi->pi", H)
    gk, uk = kept(g, how, dtype), kept(u, how, dtype)
    du = (dh * silu(gk)).round(dtype)
    dg = (dh * uk * (silu(gk) if mistake == "silu for its slope" else slope(gk))).round(dtype)
    hb = (silu(gk) * uk).round(dtype)
    drows = dot(dg, W[0], "pi,pih->ph", I)
    if mistake != "no gradient through up":
        drows = drows + dot(du, W[1], "pi,pih->ph", I)
    drows = V(drows.v, drows.e + 4 * E * drows.top()).round(dtype)

    def per_expert(a, b, how_):
        n = torch.zeros(Ex, *([a.v.shape[1], b.v.shape[1]]), dtype=torch.float64, device=x.device)
        r = V(n, torch.zeros_like(n))
        for e in range(Ex):
            on = (pair == e).nonzero()[:, 0]
            if len(on):
                d = dot(a.map(lambda t: t[on]), b.map(lambda t: t[on]), how_, len(on))
                r.v[e], r.e[e] = d.v, d.e
        return r.round(dtype)

    dgate, dup = per_expert(dg, rows, "pi,ph->ih"), per_expert(du, rows, "pi,ph->ih")
    ddown = per_expert(dy, hb, "ph,pi->hi")

    dx_rows = total(by_token(drows), 1, k + 1) + V(dx_in.double())
    if mistake == "no dx_in":
        dx_rows = total(by_token(drows), 1, k + 1)
    dx_rows = V(dx_rows.v, dx_rows.e + (k + 3) * E * dx_rows.top()).round(dtype)
    mean = total(wt * dw, 1, k).map(lambda t: t[:, None])
    if mistake == "softmax without its mean":
        mean = V(torch.zeros_like(mean.v))
    dl = wt * V(dw.v - mean.v, dw.e + mean.e + E * (dw.top() + mean.top()))
    through = dl.map(lambda t: t[:, :, None]) * V(wr[ids])
    dx = dx_rows if mistake == "no gradient through the router" else dx_rows + total(through, 1, k + 1)
    dx = V(dx.v, dx.e + (k + 3) * E * dx.top()).round(dtype)
    flat = dl.map(lambda t: t.reshape(-1))
    dwr, db = V(torch.zeros_like(wr)), V(torch.zeros(Ex, dtype=torch.float64, device=x.device))
    for e in range(Ex):
        on = (pair == e).nonzero()[:, 0]
        if len(on):
            d = flat.map(lambda t: t[on])
            r = dot(d, rows.map(lambda t: t[on]), "p,ph->h", len(on))
            s = total(d, 0, len(on))
            dwr.v[e], dwr.e[e], db.v[e], db.e[e] = r.v, r.e, s.v, s.e
    return dict(out=out, dx=dx, dwr=dwr.round(torch.float32), db=db.round(torch.float32), dgate=dgate, dup=dup,
                ddown=ddown)
