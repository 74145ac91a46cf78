"""64-bit definitions of the operators around the routed experts, with bounds
on the error of a float32 computation rounded once at the end (not a test
module).

Every function returns {name: (value, bound)}: the float64 value of an output
and the largest error a correct kernel can make.  The bounds count roundings:
e = 2^-24 for each float32 operation, u = eps / 2 of the output type for the
final rounding, relative to the magnitudes that are added.  A row sum of H
terms goes through a chain of at most H / 64 + 32 additions (64 or more threads
per row, then a tree), whatever the kernel's shape.  An underflow of float32
adds at most 2^-126 for each product (TINY, times the number of terms)."""
from __future__ import annotations

import torch

E = 2.0 ** -24
TINY = 2.0 ** -120
GATE_TOKEN, GATE_FULL, SIGMOID, NO_NORM = 1, 2, 4, 8


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def chain(H):
    return H / 64 + 32


def _norm(z, ez, w, eps):
    """norm(z) with per-element input error ez: (value, error)."""
    H = z.shape[1]
    ss = (z * z).sum(1, keepdim=True)
    ms = ss / H + eps
    rs = ms ** -0.5
    # relative error of rs: half that of the mean square
    rel = ((z.abs() * ez).sum(1, keepdim=True) / H / ms) + (chain(H) / 2 + 4) * E
    b = z * rs * w
    return b, (rs * w).abs() * ez + b.abs() * (rel + 5 * E)


def _gate(flags, gate, T):
    if not flags & (GATE_TOKEN | GATE_FULL):
        return None, None, 0.0          # factor, slope, relative error
    raw = gate.double().reshape(T, -1)
    if flags & SIGMOID:
        G = 1 / (1 + torch.exp(-raw))
        # exp2 of the rounded product g log2(e): half an ulp of an argument up to
        # 1.45 |g| changes the exponential by at most |g| e relative to its value,
        # then exp2, the addition and the reciprocal: 8 e
        return G, torch.exp(-raw) * G * G, (8 + raw.abs()) * E
    return raw, torch.ones_like(raw), 0.0


def norm_out(z, ez, w, gate, residual, w_next, *, dtype, eps, offset, rscale, bscale, flags):
    """out and n_next of a branch z (float64) known to ez."""
    T = z.shape[0]
    b, eb = z, ez
    if not flags & NO_NORM:
        b, eb = _norm(z, ez, w.double() + offset, eps)
    G, _, eg = _gate(flags, gate, T)
    if G is not None:
        eb = eb * G.abs() + (b * G).abs() * (eg + E)
        b = b * G
    v, ev = bscale * b, abs(bscale) * eb + (bscale * b).abs() * E
    if residual is not None:
        r = rscale * residual.double()
        v = v + r
        ev = ev + v.abs() * E + r.abs() * E
    res = {"out": (v, ev + v.abs() * u_of(dtype) + TINY)}
    if w_next is not None:
        n, en = _norm(v, ev, w_next.double() + offset, eps)
        res["n_next"] = (n, en + n.abs() * u_of(dtype) + TINY)
    return res


def norm_in(x, w, *, dtype, eps, offset):
    n, en = _norm(x.double(), torch.zeros_like(x, dtype=torch.float64), w.double() + offset, eps)
    return {"n": (n, en + n.abs() * u_of(dtype) + TINY)}


def norm_bwd(dout, z, w, gate, dres, *, dtype, eps, offset, rscale, bscale, flags):
    """dz, dw, dgate of norm_out (norm_in: no gate, bscale 1, dres added)."""
    z, T, H = z.double(), z.shape[0], z.shape[1]
    L = chain(H)
    normed = not flags & NO_NORM
    db = bscale * dout.double()
    W = w.double() + offset if normed else torch.ones(H, dtype=torch.float64, device=z.device)
    ms = (z * z).mean(1, keepdim=True) + eps
    rs = ms ** -0.5 if normed else torch.ones_like(ms)
    rel = (L / 2 + 4) * E if normed else 0.0
    G, slope, eg = _gate(flags, gate, T)
    G1 = torch.ones_like(ms) if G is None else G
    g = db * G1 * W
    zh = z * rs
    res = {}
    dz, edz = g, g.abs() * (5 * E + eg)
    if normed:
        c = (g * zh).mean(1, keepdim=True)
        ec = ((g * zh).abs() * ((L + 10) * E + eg + rel)).mean(1, keepdim=True)
        dz = rs * (g - zh * c)
        mag = rs * (g.abs() + (zh * c).abs())
        edz = mag * (8 * E + eg + 2 * rel) + rs * zh.abs() * ec
        t = db * G1 * zh
        # rows of a workgroup one after the other, then the workgroups
        res["dw"] = (t.sum(0), (t.abs() * ((T + 8) * E + eg + rel)).sum(0) + TINY * T)
    if dres is not None:
        d = rscale * dres.double()
        dz, edz = dz + d, edz + (dz + d).abs() * E + d.abs() * E
    res["dz"] = (dz, edz + dz.abs() * u_of(dtype) + TINY)
    if G is not None:
        t = db * zh * W * slope
        rd = (10 * E + 2 * eg + rel)
        # 1 - G is computed from the rounded G: an absolute error of e
        edge = (db * zh * W).abs() * G1.abs() * (2 * E) if flags & SIGMOID else 0.0
        if flags & GATE_TOKEN:
            val = t.sum(1)
            err = (t.abs() * ((L + 4) * E + rd)).sum(1) + (edge.sum(1) if flags & SIGMOID else 0.0)
            res["dgate"] = (val, err + TINY * H)
        else:
            res["dgate"] = (t, t.abs() * (rd + u_of(dtype)) + edge + TINY)
    return res


def _rows(pair_row, T, k):
    r = pair_row.long().reshape(T, k)
    return r, (r >= 0) & (r < T * k)


def combine(y, pair_row, topk_w, T, k):
    """(z, error) of the weighted sum of a token's slots."""
    r, on = _rows(pair_row, T, k)
    z = torch.zeros((T, y.shape[1]), dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(z)
    for j in range(k):
        i = on[:, j]
        t = topk_w[i, j, None].double() * y[r[i, j]].double()
        z[i] += t
        mag[i] += t.abs()
    return z, mag * (k * E) + TINY


def dispatch(x, pair_row, topk_w, old, *, dtype):
    """rows over `old`, what the buffer held before."""
    T, H = x.shape
    k = pair_row.numel() // T
    r, on = _rows(pair_row, T, k)
    rows, err = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    for j in range(k):
        i = on[:, j]
        v = x[i].double()
        if topk_w is not None:
            v = v * topk_w[i, j, None].double()
            err[r[i, j]] = v.abs() * (E + u_of(dtype)) + TINY
        rows[r[i, j]] = v
    return {"rows": (rows, err)}


def dispatch_bwd(drows, pair_row, topk_w, x, dx_in, T, *, dtype, dw):
    H = drows.shape[1]
    k = pair_row.numel() // T
    r, on = _rows(pair_row, T, k)
    dx = torch.zeros((T, H), dtype=torch.float64, device=drows.device)
    mag = torch.zeros_like(dx)
    gw = torch.zeros((T, k), dtype=torch.float64, device=drows.device)
    gm = torch.zeros_like(gw)
    for j in range(k):
        i = on[:, j]
        d = drows[r[i, j]].double()
        t = d if topk_w is None else topk_w[i, j, None].double() * d
        dx[i] += t
        mag[i] += t.abs()
        if dw:
            p = d * x[i].double()
            gw[i, j], gm[i, j] = p.sum(1), p.abs().sum(1)
    if dx_in is not None:
        dx, mag = dx + dx_in.double(), mag + dx_in.double().abs()
    res = {"dx": (dx, mag * ((k + 1) * E) + dx.abs() * u_of(dtype) + TINY)}
    if dw:
        res["dw"] = (gw, gm * ((chain(H) + 2) * E) + TINY * H)
    return res


def combine_bwd(dout, y, pair_row, topk_w, old, *, dtype, dw):
    T, H = dout.shape
    k = pair_row.numel() // T
    r, on = _rows(pair_row, T, k)
    dy, err = old.double().clone(), torch.zeros_like(old, dtype=torch.float64)
    gw = torch.zeros((T, k), dtype=torch.float64, device=dout.device)
    gm = torch.zeros_like(gw)
    for j in range(k):
        i = on[:, j]
        v = dout[i].double() * topk_w[i, j, None].double()
        dy[r[i, j]] = v
        err[r[i, j]] = v.abs() * (E + u_of(dtype)) + TINY
        if dw:
            p = dout[i].double() * y[r[i, j]].double()
            gw[i, j], gm[i, j] = p.sum(1), p.abs().sum(1)
    res = {"dy": (dy, err)}
    if dw:
        res["dw"] = (gw, gm * ((chain(H) + 2) * E) + TINY * H)
    return res


def route_bwd(ids, topk_w, dw, n_experts):
    w, d = topk_w.double(), dw.double()
    T, k = w.shape
    s = (w * d).sum(1, keepdim=True)
    es = (w * d).abs().sum(1, keepdim=True) * ((k / 64 + 10) * E)
    v = w * (d - s)
    ev = w.abs() * (es + 3 * E * (d.abs() + s.abs()))
    out = torch.zeros((T, n_experts), dtype=torch.float64, device=w.device)
    err = torch.zeros_like(out)
    i = ids.long()
    ok = (i >= 0) & (i < n_experts)
    t = torch.arange(T, device=w.device)[:, None].expand(T, k)
    out[t[ok], i[ok]] = v[ok]
    err[t[ok], i[ok]] = ev[ok] + TINY
    return {"dlogits": (out, err)}


def check(got, want, what=""):
    """Every output of `got` within its bound of `want` (names must agree)."""
    for name, (ref, bound) in want.items():
        g = got[name].double()
        assert g.shape == ref.shape, (what, name, g.shape, ref.shape)
        if not ref.numel():
            continue
        assert torch.isfinite(g).all(), f"{what} {name}: non-finite values"
        over = (g - ref).abs() - bound
        i = int(over.argmax())
        assert float(over.max()) <= 0, (
            f"{what} {name}: {float(g.reshape(-1)[i])} for {float(ref.reshape(-1)[i])}, "
            f"bound {float(torch.as_tensor(bound).expand_as(ref).reshape(-1)[i])}, at {i} "
            f"({int((over > 0).sum())} of {over.numel()} over)")
