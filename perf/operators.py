"""Measured calls of the operators around the routed experts: the norms before
and after the block (with its gate, its residual scale and the next block's
norm), the dispatch of token rows to expert order, the combine with the norm
after it, and their gradients.

Formulas (row t of T tokens, feature h of H, pair p = t*k + j, row r =
pair_row[p]; a pair whose pair_row is outside [0, T*k) is dropped):

  norm(v)[h]   = v[h] * rs(v) * (w[h] + offset),  rs(v) = (mean_h v[h]^2 + eps)^-1/2
  norm_in      n = norm(x)
  norm_out     out = residual_scale * residual + branch_scale * G * norm(z),
               G = gate or sigmoid(gate), one per token or one per element;
               n_next = norm_next(out)
  combine_norm z[t] = sum_j topk_w[p] y[r], then norm_out
  dispatch     rows[r] = x[t], or topk_w[p] x[t]
  gradients    of each for a given gradient of its output, and of the
               renormalized route weights with respect to the router logits:
               dlogits[t][ids_j] = w_j (dw_j - sum_i w_i dw_i), 0 elsewhere.

``own`` selects what ``run`` computes with: elementary torch operations in
float32, or the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

_DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def _norm_in(name, T, H, act, direction, dres=False, offset=0.0):
    return dict(name=name, kind="norm_in", T=T, H=H, act=act, direction=direction, dres=dres,
                offset=offset)


def _norm_out(name, T, H, act, direction, gate="none", sigmoid=False, post=True, nxt=True,
              residual=True, offset=0.0, rscale=1.0, bscale=1.0):
    return dict(name=name, kind="norm_out", T=T, H=H, act=act, direction=direction, gate=gate,
                sigmoid=sigmoid, post=post, next=nxt, residual=residual, offset=offset,
                rscale=rscale, bscale=bscale)


def _combine_norm(name, T, H, E, k, act, gate="none", sigmoid=False, post=True, nxt=True,
                  residual=True, offset=0.0, rscale=1.0, bscale=1.0, zipf=0.0, drop=0.0):
    return dict(name=name, kind="combine_norm", T=T, H=H, E=E, k=k, act=act, gate=gate,
                sigmoid=sigmoid, post=post, next=nxt, residual=residual, offset=offset,
                rscale=rscale, bscale=bscale, zipf=zipf, drop=drop)


def _dispatch(name, T, H, E, k, act, direction, weighted=False, zipf=0.0, drop=0.0):
    return dict(name=name, kind="dispatch", T=T, H=H, E=E, k=k, act=act, direction=direction,
                weighted=weighted, zipf=zipf, drop=drop)


def _combine_grad(name, T, H, E, k, act, zipf=0.0, drop=0.0):
    return dict(name=name, kind="combine_grad", T=T, H=H, E=E, k=k, act=act, zipf=zipf, drop=drop)


def listed():
    return [
        # one token of a decode loop: the norm before the routed experts
        _norm_in("norm_in_decode", 1, 2560, "bf16", "fwd"),
        # eight merged prefill windows in training: the same norm's gradient, added to the
        # gradient that arrives over the residual path
        _norm_in("norm_in_grad_merged", 32768, 2560, "bf16", "bwd", dres=True),
        # a verifier block of 16 tokens: norm after the block with a sigmoid gate per token,
        # residual add and the next block's norm
        _norm_out("norm_out_verify", 16, 2560, "bf16", "fwd", gate="token", sigmoid=True),
        # one prefill window in training, forward and gradient, a gate per element
        _norm_out("norm_out_train", 4096, 2560, "bf16", "both", gate="full", sigmoid=True,
                  bscale=0.5),
        # float32 and a width that no vector length divides, linear token gate, weights
        # stored as an offset from one
        _norm_out("norm_out_grad_odd", 777, 1001, "f32", "bwd", gate="token", offset=1.0,
                  rscale=0.75, bscale=1.25),
        # the decode batch: experts' outputs combined, residual add and the next norm (a
        # block without a norm after it)
        _combine_norm("combine_norm_decode", 8, 2560, 512, 10, "bf16", post=False),
        # one layer of the 512-token stack: combine, norm after, residual, next norm
        _combine_norm("combine_norm_stack", 512, 2560, 512, 10, "bf16", bscale=0.7),
        # the tiny float32 layer, forward and gradient of the sorted rows
        _dispatch("dispatch_tiny", 16, 256, 16, 2, "f32", "both"),
        # one prefill window under skewed routing: rows for the experts
        _dispatch("dispatch_prefill", 4096, 2560, 512, 10, "bf16", "fwd", zipf=1.1),
        # its gradient where route weights multiply the experts' inputs
        _dispatch("dispatch_grad_weighted", 4096, 2560, 512, 10, "bf16", "bwd", weighted=True,
                  zipf=1.1),
        # one prefill window in training: gradient of the weighted sum down to the logits
        _combine_grad("combine_grad_prefill", 4096, 2560, 512, 10, "bf16", zipf=1.1),
        # a ragged float32 batch in which an expert capacity dropped a tenth of the pairs
        _combine_grad("combine_grad_ragged", 333, 384, 60, 3, "f32", drop=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    kind = rng.choice(["norm_in", "norm_out", "combine_norm", "dispatch", "combine_grad"])
    act = rng.choice(["bf16", "bf16", "f32"])
    gate = rng.choice(["none", "token", "full"])
    out = dict(gate=gate, sigmoid=gate != "none" and rng.random() < 0.5,
               post=rng.random() < 0.7, nxt=rng.random() < 0.7, residual=rng.random() < 0.8,
               offset=rng.choice([0.0, 1.0]), rscale=rng.choice([1.0, 0.5]),
               bscale=rng.choice([1.0, 0.22]))
    if kind in ("norm_in", "norm_out"):
        T = _log_int(rng, 1, 32768)
        H = rng.choice([_log_int(rng, 33, 8191), 8 * _log_int(rng, 8, 1024), 2560])
        direction = rng.choice(["fwd", "bwd", "both"])
        if kind == "norm_in":
            make = lambda t: _norm_in("", t, H, act, direction, dres, out["offset"])
            dres = rng.random() < 0.5
        else:
            make = lambda t: _norm_out("", t, H, act, direction, **out)
    else:
        T = _log_int(rng, 1, 4096)
        H = rng.choice([128 * rng.randint(1, 56), 2560])
        E = rng.choice([_log_int(rng, 2, 1024), 512])
        k = min(E, rng.randint(1, 16))
        route = dict(zipf=rng.choice([0.0, 1.1]), drop=rng.choice([0.0, 0.0, 0.1]))
        if kind == "combine_norm":
            make = lambda t: _combine_norm("", t, H, E, k, act, **out, **route)
        elif kind == "dispatch":
            direction, weighted = rng.choice(["fwd", "bwd", "both"]), rng.random() < 0.5
            make = lambda t: _dispatch("", t, H, E, k, act, direction, weighted, **route)
        else:
            make = lambda t: _combine_grad("", t, H, E, k, act, **route)
    while work(make(T))["bytes"] > most:
        T = max(1, T * 3 // 4)
    case = make(T)
    del case["name"]
    return case


def _gate_bytes(c, a):
    n = c["T"] * c["H"] * a
    return {"none": 0, "token": 4 * c["T"], "full": n}[c["gate"]]


def work(case):
    c = case
    T, H = c["T"], c["H"]
    a = 2 if c["act"] == "bf16" else 4
    n, row = T * H * a, H * a
    kind = c["kind"]
    b = f = 0
    if kind == "norm_in":
        if c["direction"] != "bwd":
            b += 2 * n + row                                   # x, w -> n
            f += 4 * T * H
        if c["direction"] != "fwd":
            b += (4 if c["dres"] else 3) * n + row + 4 * H     # dn, x, w (, dres) -> dx, dw
            f += 10 * T * H
    elif kind in ("norm_out", "combine_norm"):
        g = _gate_bytes(c, a)
        if kind == "combine_norm" or c["direction"] != "bwd":
            b += n + g + (n if c["residual"] else 0)           # (z), gate, residual -> out
            f += 8 * T * H
            b += row if c["post"] else 0
            if c["next"]:
                b += n + row
                f += 4 * T * H
            if kind == "norm_out":
                b += n
            else:
                b += c["k"] * (n + 8 * T)                      # y, pair_row, topk_w
                f += 2 * c["k"] * T * H
        if kind == "norm_out" and c["direction"] != "fwd":
            b += 2 * n + g                                     # dout, gate -> dz
            f += 14 * T * H
            if c["gate"] != "none" or c["post"]:
                b += n + g                                     # z; dgate
            if c["post"]:
                b += row + 4 * H                               # w; dw
    elif kind == "dispatch":
        k, w = c["k"], 4 * T * c["k"]
        if c["direction"] != "bwd":
            b += n + k * n + w + (w if c["weighted"] else 0)   # x, pair_row (, topk_w) -> rows
            f += k * T * H if c["weighted"] else 0
        if c["direction"] != "fwd":
            b += k * n + n + w + ((n + 2 * w) if c["weighted"] else 0)
            f += k * T * H * (4 if c["weighted"] else 1)
    else:
        k, w = c["k"], 4 * T * c["k"]
        b += n + 2 * k * n + 4 * w + 4 * T * c["E"]            # dout, y, rows, w, ids -> dy, dw, dlogits
        f += 3 * k * T * H
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    c, dt = case, _TYPES[case["act"]]
    T, H = c["T"], c["H"]
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)

    def normal(shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=_DEV) * std + mean).to(dtype)

    d = {}
    kind = c["kind"]
    if kind == "norm_in":
        d["x"], d["w"] = normal((T, H)), normal((H,), 0.1, 1.0 - c["offset"])
        if c["direction"] != "fwd":
            d["dn"] = normal((T, H), 0.1)
            d["dres"] = normal((T, H), 0.1) if c["dres"] else None
        return d
    if kind in ("norm_out", "combine_norm"):
        d["w"] = normal((H,), 0.1, 1.0 - c["offset"]) if c["post"] else None
        d["w_next"] = normal((H,), 0.1, 1.0 - c["offset"]) if c["next"] else None
        d["gate"] = {"none": lambda: None, "token": lambda: normal((T,), dtype=torch.float32),
                     "full": lambda: normal((T, H))}[c["gate"]]()
        d["residual"] = normal((T, H), 1.5) if c["residual"] else None
    if kind == "norm_out":
        d["z"] = normal((T, H), 0.3)
        if c["direction"] != "fwd":
            d["dout"] = normal((T, H), 0.1)
        return d
    # routes: the k best of skewed random logits, renormalized weights, pairs sorted by expert
    E, k = c["E"], c["k"]
    P = T * k
    logits = torch.randn((T, E), generator=g, device=_DEV)
    if c["zipf"]:
        rank = torch.arange(1, E + 1, device=_DEV, dtype=torch.float32)
        logits = logits - 0.5 * c["zipf"] * torch.log(rank)
    top, ids = torch.topk(logits, k, dim=1)
    d["topk_ids"] = ids.to(torch.int32).contiguous()
    d["topk_w"] = torch.softmax(top, dim=1).contiguous()
    order = torch.argsort(ids.reshape(-1), stable=True)
    row = torch.empty(P, dtype=torch.int64, device=_DEV)
    row[order] = torch.arange(P, device=_DEV)
    if c["drop"]:
        row[torch.rand(P, generator=g, device=_DEV) < c["drop"]] = -1
    d["pair_row"] = row.to(torch.int32)
    if kind == "combine_norm":
        d["y"] = normal((P, H), 0.3)
    elif kind == "dispatch":
        d["x"] = normal((T, H))
        if c["direction"] != "fwd":
            d["drows"] = normal((P, H), 0.1)
    else:
        d["dout"], d["y"] = normal((T, H), 0.1), normal((P, H), 0.3)
    return d


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own:
        _own_buffers(state)
    return state


def _own_buffers(s):
    """Descriptors, outputs and workspace that a program keeps for a shape."""
    import sparse_moe_routed_amd as M
    c = s["case"]
    dt, T, H, kind = _TYPES[c["act"]], c["T"], c["H"], c["kind"]
    new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=_DEV)
    if "k" in c:
        s["shape"] = M.make_shape(T, H, c["E"], 128, c["k"], c["act"])
        P = T * c["k"]
    if kind in ("norm_in", "norm_out", "combine_norm"):
        flags = 0
        if kind != "norm_in":
            flags = {"none": 0, "token": M.MOE_N_GATE_TOKEN, "full": M.MOE_N_GATE_FULL}[c["gate"]]
            flags |= M.MOE_N_GATE_SIGMOID if c["sigmoid"] else 0
            flags |= 0 if c["post"] else M.MOE_N_NO_NORM
        s["norm"] = M.make_norm(T, H, c["act"], eps=_EPS, weight_offset=c["offset"],
                                residual_scale=c.get("rscale", 1.0),
                                branch_scale=c.get("bscale", 1.0), flags=flags)
        s["ws_bytes"] = M.moe_norm_workspace_size(s["norm"])
        s["ws"] = torch.empty(max(s["ws_bytes"], 1), dtype=torch.uint8, device=_DEV)
    if kind == "norm_in":
        s.update(n=new(T, H), dx=new(T, H), dw=new(H, dtype=torch.float32))
    elif kind in ("norm_out", "combine_norm"):
        s.update(out=new(T, H), n_next=new(T, H) if c["next"] else None, dz=new(T, H),
                 dw=new(H, dtype=torch.float32) if c["post"] else None,
                 dgate=None if s["gate"] is None else torch.empty_like(s["gate"]))
    elif kind == "dispatch":
        s.update(rows=new(P, H), dx=new(T, H),
                 dw=new(T, c["k"], dtype=torch.float32) if c["weighted"] else None)
    else:
        s.update(dy=new(P, H), dw=new(T, c["k"], dtype=torch.float32),
                 dlogits=new(T, c["E"], dtype=torch.float32))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(state):
    return dict(sorted((_run_own if own else _run_plain)(state).items()))


def _run_own(s):
    import sparse_moe_routed_amd as M
    c, kind, res = s["case"], s["case"]["kind"], {}
    if kind == "norm_in":
        if c["direction"] != "bwd":
            M.moe_norm_in(s["norm"], s["x"], s["w"], s["n"])
            res["n"] = s["n"]
        if c["direction"] != "fwd":
            M.moe_norm_in_backward(s["norm"], s["dn"], s["x"], s["w"], s["dres"], s["dx"], s["dw"],
                                   s["ws"], s["ws_bytes"])
            res.update(dx=s["dx"], dw=s["dw"])
    elif kind == "norm_out":
        if c["direction"] != "bwd":
            M.moe_norm_out(s["norm"], s["z"], s["w"], s["gate"], s["residual"], s["w_next"],
                           s["out"], s["n_next"])
            res["out"] = s["out"]
            if c["next"]:
                res["n_next"] = s["n_next"]
        if c["direction"] != "fwd":
            M.moe_norm_out_backward(s["norm"], s["dout"], s["z"], s["w"], s["gate"], s["dz"],
                                    s["dgate"], s["dw"], s["ws"], s["ws_bytes"])
            res["dz"] = s["dz"]
            if c["gate"] != "none":
                res["dgate"] = s["dgate"]
            if c["post"]:
                res["dw"] = s["dw"]
    elif kind == "combine_norm":
        M.moe_combine_norm(s["shape"], s["norm"], s["y"], s["pair_row"], s["topk_w"], s["w"],
                           s["gate"], s["residual"], s["w_next"], None, s["out"], s["n_next"])
        res["out"] = s["out"]
        if c["next"]:
            res["n_next"] = s["n_next"]
    elif kind == "dispatch":
        w = s["topk_w"] if c["weighted"] else None
        if c["direction"] != "bwd":
            if c["drop"]:
                s["rows"].zero_()              # rows that no pair names
            M.moe_dispatch(s["shape"], s["x"], s["pair_row"], w, s["rows"])
            res["rows"] = s["rows"]
        if c["direction"] != "fwd":
            M.moe_dispatch_backward(s["shape"], s["drows"], s["pair_row"], w,
                                    s["x"] if c["weighted"] else None, None, s["dx"], s["dw"])
            res["dx"] = s["dx"]
            if c["weighted"]:
                res["dw"] = s["dw"]
    else:
        if c["drop"]:
            s["dy"].zero_()                    # rows that no pair names
        M.moe_combine_backward(s["shape"], s["dout"], s["y"], s["pair_row"], s["topk_w"], s["dy"],
                               s["dw"])
        M.moe_route_backward(s["shape"], s["topk_ids"], s["topk_w"], s["dw"], s["dlogits"])
        res.update(dy=s["dy"], dw=s["dw"], dlogits=s["dlogits"])
    return res


def _rs(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS)


def _out_plain(c, s, z):
    """The block's output and the next norm, float32, from its branch z."""
    dt = _TYPES[c["act"]]
    v = z
    if c["post"]:
        v = v * _rs(v) * (s["w"].float() + c["offset"])
    if c["gate"] != "none":
        G = s["gate"].float()
        G = torch.sigmoid(G) if c["sigmoid"] else G
        v = v * (G[:, None] if c["gate"] == "token" else G)
    v = v * c["bscale"]
    if c["residual"]:
        v = v + s["residual"].float() * c["rscale"]
    res = {"out": v.to(dt)}
    if c["next"]:
        res["n_next"] = (v * _rs(v) * (s["w_next"].float() + c["offset"])).to(dt)
    return res


def _run_plain(s):
    c, kind, res = s["case"], s["case"]["kind"], {}
    dt, T, H = _TYPES[c["act"]], c["T"], c["H"]
    if kind == "norm_in":
        x, w = s["x"].float(), s["w"].float() + c["offset"]
        xh = x * _rs(x)
        if c["direction"] != "bwd":
            res["n"] = (xh * w).to(dt)
        if c["direction"] != "fwd":
            dn = s["dn"].float()
            gx = dn * w
            dx = _rs(x) * (gx - xh * (gx * xh).mean(dim=1, keepdim=True))
            if s["dres"] is not None:
                dx = dx + s["dres"].float()
            res.update(dx=dx.to(dt), dw=(dn * xh).sum(dim=0))
        return res
    if kind == "norm_out":
        z = s["z"].float()
        if c["direction"] != "bwd":
            res.update(_out_plain(c, s, z))
        if c["direction"] != "fwd":
            db = s["dout"].float() * c["bscale"]
            zh, w = z, 1.0
            if c["post"]:
                zh, w = z * _rs(z), s["w"].float() + c["offset"]
            if c["gate"] != "none":
                G = s["gate"].float()
                slope = 1.0
                if c["sigmoid"]:
                    G = torch.sigmoid(G)
                    slope = G * (1.0 - G)
                dG = db * zh * w
                dG = dG.sum(dim=1) if c["gate"] == "token" else dG
                res["dgate"] = (dG * slope).to(s["gate"].dtype)
                db = db * (G[:, None] if c["gate"] == "token" else G)
            if c["post"]:
                res["dw"] = (db * zh).sum(dim=0)
                gz = db * w
                db = _rs(z) * (gz - zh * (gz * zh).mean(dim=1, keepdim=True))
            res["dz"] = db.to(dt)
        return res
    k, E = c["k"], c["E"]
    row = s["pair_row"].long()
    kept = (row >= 0)
    safe = row.clamp(min=0)
    keptw = kept.float().reshape(T, k)
    if kind == "combine_norm":
        z = torch.zeros((T, H), device=_DEV)
        for j in range(k):
            wj = (s["topk_w"][:, j] * keptw[:, j])[:, None]
            z = z + wj * s["y"][safe.reshape(T, k)[:, j]].float()
        return _out_plain(c, s, z)
    if kind == "dispatch":
        if c["direction"] != "bwd":
            v = s["x"].float()[:, None, :].expand(T, k, H)
            if c["weighted"]:
                v = v * s["topk_w"][:, :, None]
            rows = torch.zeros((T * k, H), dtype=dt, device=_DEV)
            rows[row[kept]] = v.reshape(T * k, H)[kept].to(dt)
            res["rows"] = rows
        if c["direction"] != "fwd":
            dv = s["drows"][safe].float().reshape(T, k, H) * keptw[:, :, None]
            if c["weighted"]:
                res["dw"] = (dv * s["x"].float()[:, None, :]).sum(dim=2)
                dv = dv * s["topk_w"][:, :, None]
            res["dx"] = dv.sum(dim=1).to(dt)
        return res
    dout = s["dout"].float()
    yk = s["y"][safe].float().reshape(T, k, H)
    dw = (yk * dout[:, None, :]).sum(dim=2) * keptw
    dy = torch.zeros((T * k, H), dtype=dt, device=_DEV)
    v = (dout[:, None, :] * s["topk_w"][:, :, None]).to(dt)
    dy[row[kept]] = v.reshape(T * k, H)[kept]
    wk = s["topk_w"]
    dl = wk * (dw - (wk * dw).sum(dim=1, keepdim=True))
    dlogits = torch.zeros((T, E), device=_DEV)
    dlogits.scatter_(1, s["topk_ids"].long(), dl)
    return {"dy": dy, "dw": dw, "dlogits": dlogits}


# ---------------------------------------------------------------------------
# Definition in 64 bits
# ---------------------------------------------------------------------------


def _branch64(c, s, z):
    """(block output, next norm) in float64."""
    b = z
    if c["post"]:
        ms = (z ** 2).sum(1) / c["H"]
        b = z / torch.sqrt(ms + _EPS)[:, None] * (c["offset"] + s["w"].double())[None, :]
    if s["gate"] is not None:
        G = s["gate"].double()
        if c["sigmoid"]:
            G = 1.0 / (1.0 + torch.exp(-G))
        b = b * G.reshape(c["T"], -1)
    out = c["bscale"] * b
    if c["residual"]:
        out = out + c["rscale"] * s["residual"].double()
    res = {"out": out}
    if c["next"]:
        ms = (out ** 2).sum(1) / c["H"]
        res["n_next"] = out / torch.sqrt(ms + _EPS)[:, None] * (c["offset"] + s["w_next"].double())
    return res


def _norm_grad64(v, w, g):
    """(dv, dw) of v / sqrt(mean v^2 + eps) * w for an output gradient g:
    dv = w g / r - v (sum_h v w g) / (H r^3) with r the root."""
    r = torch.sqrt((v ** 2).sum(1) / v.shape[1] + _EPS)
    inner = (v * g * w).sum(1)
    dv = g * w / r[:, None] - v * (inner / (v.shape[1] * r ** 3))[:, None]
    return dv, (g * (v / r[:, None])).sum(0)


def exact(case, seed):
    return dict(sorted(_exact(case, _inputs(case, seed)).items()))


def _exact(c, s):
    T, H, kind, res = c["T"], c["H"], c["kind"], {}
    D = lambda key: s[key].double()
    if kind == "norm_in":
        w = D("w") + c["offset"]
        if c["direction"] != "bwd":
            res["n"] = D("x") / torch.sqrt((D("x") ** 2).mean(1, keepdim=True) + _EPS) * w
        if c["direction"] != "fwd":
            res["dx"], res["dw"] = _norm_grad64(D("x"), w, D("dn"))
            if s["dres"] is not None:
                res["dx"] = res["dx"] + D("dres")
        return res
    if kind == "norm_out":
        if c["direction"] != "bwd":
            res.update(_branch64(c, s, D("z")))
        if c["direction"] != "fwd":
            z, go = D("z"), c["bscale"] * D("dout")
            w = D("w") + c["offset"] if c["post"] else torch.ones(H, dtype=torch.float64, device=_DEV)
            gb = go
            if s["gate"] is not None:
                raw = D("gate").reshape(T, -1)
                G = 1.0 / (1.0 + torch.exp(-raw)) if c["sigmoid"] else raw
                gb = go * G
                b = z * w
                if c["post"]:
                    b = b / torch.sqrt((z ** 2).mean(1, keepdim=True) + _EPS)
                dG = go * b
                dG = dG.sum(1, keepdim=True) if c["gate"] == "token" else dG
                if c["sigmoid"]:
                    dG = dG * torch.exp(-raw) * G * G
                res["dgate"] = dG.reshape(s["gate"].shape)
            if c["post"]:
                res["dz"], res["dw"] = _norm_grad64(z, w, gb)
            else:
                res["dz"] = gb
        return res
    k, E = c["k"], c["E"]
    rows = s["pair_row"].long().reshape(T, k)
    wk = D("topk_w")
    if kind == "combine_norm":
        z = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
        for j in range(k):
            on = rows[:, j] >= 0
            z[on] += wk[on, j, None] * s["y"][rows[on, j]].double()
        return _branch64(c, s, z)
    if kind == "dispatch":
        if c["direction"] != "bwd":
            out = torch.zeros((T * k, H), dtype=torch.float64, device=_DEV)
            for j in range(k):
                on = rows[:, j] >= 0
                v = D("x")[on]
                out[rows[on, j]] = v * wk[on, j, None] if c["weighted"] else v
            res["rows"] = out
        if c["direction"] != "fwd":
            dx = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
            dw = torch.zeros((T, k), dtype=torch.float64, device=_DEV)
            for j in range(k):
                on = rows[:, j] >= 0
                v = s["drows"][rows[on, j]].double()
                dw[on, j] = (v * D("x")[on]).sum(1)
                dx[on] += v * wk[on, j, None] if c["weighted"] else v
            res["dx"] = dx
            if c["weighted"]:
                res["dw"] = dw
        return res
    dy = torch.zeros((T * k, H), dtype=torch.float64, device=_DEV)
    dw = torch.zeros((T, k), dtype=torch.float64, device=_DEV)
    for j in range(k):
        on = rows[:, j] >= 0
        dy[rows[on, j]] = D("dout")[on] * wk[on, j, None]
        dw[on, j] = (D("dout")[on] * s["y"][rows[on, j]].double()).sum(1)
    dl = wk * dw - wk * (wk * dw).sum(1, keepdim=True)
    dlogits = torch.zeros((T, E), dtype=torch.float64, device=_DEV)
    dlogits[torch.arange(T, device=_DEV)[:, None], s["topk_ids"].long()] = dl
    return {"dy": dy, "dw": dw, "dlogits": dlogits}
