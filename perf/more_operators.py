"""Cases of the framework's layers around the linear one: the embedding lookup and its gradient by
sorted tokens, layer norm forward and backward, the gated feed-forward projections forward and
backward, and the loss against targets and a teacher's top logits with its gradient.

``run`` computes a case either in plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where ``own`` is true, by the framework's calls.  ``exact`` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
SCALE = 1.5  # of the embedding
GRAD_SCALE = 8.0  # of the loss: a loss scale over the number of tokens


def listed():
    return [
        # the tokens of a training batch looked up in the 1.3e9-parameter workload's table
        dict(name="embed-16k", op="embed", t=16384, d=2048, v=44629, type="bf16", pad=0),
        # their gradient: every row of the table's gradient is written
        dict(name="embed-grad-16k", op="embed_grad", t=16384, d=2048, v=44629, add=False, type="bf16", pad=0),
        # a table shared with the output layer, whose gradient is there already; odd sizes
        dict(name="embed-grad-odd", op="embed_grad", t=1009, d=331, v=10007, add=True, type="fp16", pad=1),
        # a few tokens through a norm: latency of a call
        dict(name="norm-4tokens", op="norm", t=4, d=2048, type="bf16", pad=0),
        # a training batch's norm, backward, with the gradient that passes by on the residual
        dict(name="norm-grad-16k", op="norm_grad", t=16384, d=2048, residual=True, type="bf16", pad=0),
        # odd width, rows off the 16-byte boundary
        dict(name="norm-grad-odd", op="norm_grad", t=1009, d=1001, residual=False, type="fp16", pad=3),
        # a few tokens through the two projections (generation, tiny batches)
        dict(name="gated-4tokens", op="gated", t=4, k=2048, n=8192, act="silu", keep=False, bias=False, type="bf16", pad=0),
        # a training batch's, with what the backward pass needs
        dict(name="gated-8k", op="gated", t=8192, k=2048, n=8192, act="silu", keep=True, bias=False, type="bf16", pad=0),
        # odd sizes and rows off the 16-byte boundary
        dict(name="gated-odd", op="gated", t=509, k=777, n=1190, act="gelu", keep=True, bias=True, type="fp16", pad=1),
        # the gradients of a training batch's projections
        dict(name="gated-grad-8k", op="gated_grad", t=8192, k=2048, n=8192, act="silu", bias=True, type="bf16", pad=0),
        # a small model's loss against a teacher's 20 logits, odd vocabulary, a quarter of it masked
        dict(name="distill-odd", op="distill", t=509, v=10007, k=20, tau=1.0, alpha=0.9, masked=2500, teacher="fp32", type="fp16", pad=0),
        # a training batch's loss, half from the targets, half from a teacher's 64 logits
        dict(name="distill-8k", op="distill", t=8192, v=44629, k=64, tau=2.0, alpha=0.5, masked=0, teacher="bf16", type="bf16", pad=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: any, or a multiple of 64 as models have them."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.5 else max(64, w // 64 * 64)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "gated", "gated_grad", "distill"])
    c = dict(op=op, type=rng.choice(["fp16", "bf16"]), pad=rng.choice([0, 0, 1, 8]))
    if op in ("embed", "embed_grad"):
        d = _width(rng, 40, 4096)
        v = min(_log(rng, 100, 200000), 44629 * 2048 // d)
        c.update(t=min(_log(rng, 1, 65536), 16384 * 2048 // d), d=d, v=v)
        if op == "embed_grad":
            c["add"] = rng.random() < 0.4
    elif op in ("norm", "norm_grad"):
        d = _width(rng, 16, 16384)
        c.update(t=min(_log(rng, 1, 65536), 16384 * 2048 // d), d=d)
        if op == "norm_grad":
            c["residual"] = rng.random() < 0.5
    elif op in ("gated", "gated_grad"):
        k, n = _width(rng, 64, 4096), _width(rng, 64, 8192)
        t = max(1, min(_log(rng, 1, 16384), 8192 * 2048 * 8192 // (k * n)))
        c.update(t=t, k=k, n=n, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5)
        if op == "gated":
            c["keep"] = rng.random() < 0.5
    else:
        v = _log(rng, 200, 150000)
        t = min(_log(rng, 1, 16384), 8192 * 44629 // v)
        c.update(t=t, v=v, k=rng.choice([0, 1, 8, 20, 50, 64, 100]), tau=rng.choice([1.0, 1.0, 1.5, 2.0, 4.0]), alpha=rng.choice([0.0, 0.5, 0.9, 1.0]),
                 masked=rng.choice([0, 0, v // 4]), teacher=rng.choice(["fp16", "bf16", "fp32"]))
        if c["k"] == 0:
            c["alpha"] = 0.0
    return c


# ---------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------


def _distinct(t, v):
    """Rows of the table that t tokens with probabilities in proportion to log((i + 2) / (i + 1)) are expected to name."""
    i = np.arange(v, dtype=np.float64)
    p = np.log((i + 2) / (i + 1)) / math.log(v + 1)
    return float((1 - (1 - p) ** t).sum())


def work(c):
    op, t = c["op"], c["t"]
    if op == "embed":
        return {"bytes": 4 * t + 2 * c["d"] * (_distinct(t, c["v"]) + t), "flops": t * c["d"]}
    if op == "embed_grad":
        rows = 2 * _distinct(t, c["v"]) if c["add"] else c["v"]
        return {"bytes": 4 * t + 2 * c["d"] * (t + rows), "flops": t * c["d"]}
    if op == "norm":
        return {"bytes": 4 * t * c["d"] + 8 * t + 4 * c["d"], "flops": 8 * t * c["d"]}
    if op == "norm_grad":
        return {"bytes": 2 * t * c["d"] * (3 + c["residual"]) + 8 * t + 6 * c["d"], "flops": 14 * t * c["d"]}
    if op == "distill":
        teacher = (4 + (4 if c["teacher"] == "fp32" else 2)) * c["k"] if c["alpha"] > 0 else 0
        return {"bytes": t * (4 * c["v"] + teacher + 12), "flops": 8 * t * c["v"]}
    k, n = c["k"], c["n"]
    if op == "gated":
        moved = t * k + 2 * n * k + 2 * n * c["bias"] + t * n * (3 if c["keep"] else 1)
        return {"bytes": 2 * moved, "flops": 4 * t * k * n}
    return {"bytes": 2 * (3 * t * n + 2 * t * k + 4 * n * k + 2 * n * c["bias"]), "flops": 8 * t * k * n}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------


def prepare(c, seed):
    s = _inputs(c, seed)
    s["case"] = c
    if own:
        _attach(s)
    return s


def _rows(t, width, pad, dtype, gen, scale, offset=0.0):
    """[t, width] values in rows of width + pad elements."""
    return (torch.randn((t, width + pad), generator=gen, device=DEV) * scale + offset).to(dtype)[:, :width]


def _room(t, width, pad, dtype):
    return torch.empty((t, width + pad), dtype=dtype, device=DEV)[:, :width]


def _tokens(t, v, gen):
    """Tokens as text has them (a few frequent, many rare ones), in an order of rows of their own; one in fifty is padding (-1)."""
    u = torch.rand(t, generator=gen, device=DEV, dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1)) - 1).long().clamp_(0, v - 1)
    ids = torch.randperm(v, generator=gen, device=DEV)[rank]
    ids[torch.rand(t, generator=gen, device=DEV) < 0.02] = -1
    return ids.int()


def _inputs(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, t, dt, pad = c["op"], c["t"], TYPES[c["type"]], c["pad"]
    if op == "embed":
        return {"ids": _tokens(t, c["v"], gen), "table": _rows(c["v"], c["d"], pad, dt, gen, 0.02), "y": _room(t, c["d"], pad, dt)}
    if op == "embed_grad":
        return {"ids": _tokens(t, c["v"], gen), "dy": _rows(t, c["d"], pad, dt, gen, 0.1), "dtable": _rows(c["v"], c["d"], pad, dt, gen, 0.1)}
    if op in ("norm", "norm_grad"):
        d = c["d"]
        s = {"x": _rows(t, d, pad, dt, gen, 1.5, 0.25), "w": (1 + 0.1 * torch.randn(d, generator=gen, device=DEV)).to(dt)}
        if op == "norm":
            s["b"] = (0.1 * torch.randn(d, generator=gen, device=DEV)).to(dt)
            s.update(y=_room(t, d, pad, dt), mean=torch.empty(t, device=DEV), rstd=torch.empty(t, device=DEV))
            return s
        x = s["x"].double()  # the forward pass's statistics
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = (((x - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
        s["dy"] = _rows(t, d, pad, dt, gen, 0.1)
        s["res"] = _rows(t, d, pad, dt, gen, 0.1) if c["residual"] else None
        s.update(dx=_room(t, d, pad, dt), dw=torch.empty(d, dtype=dt, device=DEV), db=torch.empty(d, dtype=dt, device=DEV))
        return s
    if op == "distill":
        v, k = c["v"], c["k"]
        logits = _rows(t, v, pad, dt, gen, 2.0)
        allowed = v - c["masked"]
        if c["masked"]:
            logits[:, allowed:] = -math.inf
        s = {"logits": logits, "index": None, "teacher": None, "loss": torch.empty(t, device=DEV), "dlogits": _room(t, v, pad, dt)}
        first = torch.randint(allowed, (t, 1), generator=gen, device=DEV)
        if k:
            gaps = torch.randint(1, max(2, allowed // k + 1), (t, k - 1), generator=gen, device=DEV)
            s["index"] = ((torch.cat((first, gaps), 1).cumsum(1)) % allowed).int()  # all different
            s["teacher"] = (torch.randn((t, k), generator=gen, device=DEV) * 2 + 6).sort(1, descending=True).values.to(TYPES[c["teacher"]])
        targets = first[:, 0].int()
        targets[torch.rand(t, generator=gen, device=DEV) < 0.05] = -1  # tokens without a target (a prompt's)
        s["targets"] = targets
        weights = torch.rand(t, generator=gen, device=DEV) + 0.5
        weights[torch.rand(t, generator=gen, device=DEV) < 0.05] = 0.0  # padding
        s["weights"] = weights
        return s
    k, n = c["k"], c["n"]
    s = {"x": _rows(t, k, pad, dt, gen, 1.0), "wg": _rows(n, k, pad, dt, gen, 1 / math.sqrt(k)), "wu": _rows(n, k, pad, dt, gen, 1 / math.sqrt(k))}
    if op == "gated":
        for b in ("bg", "bu"):
            s[b] = (torch.randn(n, generator=gen, device=DEV) * 0.1).to(dt) if c["bias"] else None
        s["h"] = _room(t, n, pad, dt)
        for z in ("g", "u"):
            s[z] = _room(t, n, pad, dt) if c["keep"] else None
        return s
    s.update(dh=_rows(t, n, pad, dt, gen, 0.1), g=_rows(t, n, pad, dt, gen, 1.0), u=_rows(t, n, pad, dt, gen, 1.0))
    s["dx"] = _room(t, k, pad, dt)
    for w, b in (("dwg", "dbg"), ("dwu", "dbu")):
        s[w] = torch.empty((n, k), dtype=dt, device=DEV)
        s[b] = torch.empty(n, dtype=dt, device=DEV) if c["bias"] else None
    return s


def _attach(s):
    """The workspace that a program keeps for the framework's calls."""
    import zero_sharded_mixed_shard_gb300 as z

    c = s["case"]
    s["z_"], op = z, c["op"]
    types = {"fp16": z.TYPE_FP16, "bf16": z.TYPE_BF16, "fp32": z.TYPE_FP32}
    s["type"] = types[c["type"]]
    need = 0
    if op == "embed_grad":
        need = z.zero_embed_workspace(c["t"], c["d"], c["v"])
    elif op == "norm_grad":
        need = z.zero_layernorm_workspace(c["t"], c["d"])
    elif op == "distill":
        s["teacher_type"] = types[c["teacher"]]
    elif op in ("gated", "gated_grad"):
        s["act"] = {"none": z.ACT_NONE, "relu": z.ACT_RELU, "gelu": z.ACT_GELU, "silu": z.ACT_SILU}[c["act"]]
        aligned = all(s.get(m) is None or (s[m].data_ptr() % 16 == 0 and s[m].stride(0) % 8 == 0) for m in ("x", "wg", "wu"))
        need = z.zero_gated_workspace(c["t"], c["k"], c["n"], op == "gated_grad", aligned)
    s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"embed": _own_embed, "embed_grad": _own_embed_grad, "norm": _own_norm, "norm_grad": _own_norm_grad, "gated": _own_gated,
                "gated_grad": _own_gated_grad, "distill": _own_distill}[op](s)
    return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad, "gated": _plain_gated,
            "gated_grad": _plain_gated_grad, "distill": _plain_distill}[op](s)


def _ld(x):
    return 0 if x is None else x.stride(0)


def _own_embed(s):
    c, table, y = s["case"], s["table"], s["y"]
    s["z_"].zero_embed_forward(s["ids"], table, _ld(table), y, _ld(y), c["t"], c["d"], c["v"], SCALE, s["type"])
    return y


def _own_embed_grad(s):
    c, dy, dt = s["case"], s["dy"], s["dtable"]
    s["z_"].zero_embed_backward(s["ids"], dy, _ld(dy), dt, _ld(dt), c["t"], c["d"], c["v"], SCALE, c["add"], s["type"], s["ws"], s["ws"].numel())
    return dt


def _own_norm(s):
    c, x, y = s["case"], s["x"], s["y"]
    s["z_"].zero_layernorm_forward(x, _ld(x), s["w"], s["b"], y, _ld(y), s["mean"], s["rstd"], c["t"], c["d"], EPS, s["type"])
    return {"y": y, "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_grad(s):
    c, x, dy, res, dx = s["case"], s["x"], s["dy"], s["res"], s["dx"]
    s["z_"].zero_layernorm_backward(dy, _ld(dy), x, _ld(x), s["w"], s["mean"], s["rstd"], res, _ld(res), dx, _ld(dx), s["dw"], s["db"],
                                    c["t"], c["d"], s["type"], s["ws"], s["ws"].numel())
    return {"dx": dx, "dw": s["dw"], "db": s["db"]}


def _own_gated(s):
    c, x, wg, wu, h, g, u = s["case"], s["x"], s["wg"], s["wu"], s["h"], s["g"], s["u"]
    s["z_"].zero_gated_forward(x, _ld(x), wg, _ld(wg), wu, _ld(wu), s["bg"], s["bu"], h, _ld(h), g, _ld(g), u, _ld(u),
                               c["t"], c["k"], c["n"], s["act"], s["type"], s["ws"], s["ws"].numel())
    return {"h": h, "g": g, "u": u}


def _own_gated_grad(s):
    c, x, wg, wu, dh, g, u, dx = s["case"], s["x"], s["wg"], s["wu"], s["dh"], s["g"], s["u"], s["dx"]
    s["z_"].zero_gated_backward(dh, _ld(dh), g, _ld(g), u, _ld(u), x, _ld(x), wg, _ld(wg), wu, _ld(wu), dx, _ld(dx), s["dwg"], _ld(s["dwg"]),
                                s["dwu"], _ld(s["dwu"]), s["dbg"], s["dbu"], c["t"], c["k"], c["n"], s["act"], s["type"], s["ws"], s["ws"].numel())
    return {k: s[k] for k in ("dx", "dwg", "dwu", "dbg", "dbu")}


def _own_distill(s):
    c, logits, dl = s["case"], s["logits"], s["dlogits"]
    s["z_"].zero_distill_loss(logits, _ld(logits), s["targets"], s["index"], s["teacher"], _ld(s["index"]), s["weights"], s["loss"], dl, _ld(dl),
                              c["t"], c["v"], c["k"], c["tau"], c["alpha"], GRAD_SCALE, s["type"], s["teacher_type"])
    return {"loss": s["loss"], "dlogits": dl}


def _plain_embed(s):
    ids = s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * SCALE
    return torch.where((ids >= 0)[:, None], rows, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s):
    dt = s["dtable"]
    ids = s["ids"].long()
    rows = torch.where((ids >= 0)[:, None], s["dy"].float(), 0.0)
    total = torch.zeros(dt.shape, device=DEV).index_add_(0, ids.clamp(min=0), rows) * SCALE
    dt.copy_(total + dt.float() if s["case"]["add"] else total)
    return dt


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    y = x * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(s):
    dt, rstd = s["x"].dtype, s["rstd"][:, None]
    hat = (s["x"].float() - s["mean"][:, None]) * rstd
    dy = s["dy"].float()
    a = dy * s["w"].float()
    dx = rstd * (a - a.mean(1, keepdim=True) - hat * (a * hat).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(dt), "dw": (dy * hat).sum(0).to(dt), "db": dy.sum(0).to(dt)}


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        u = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-u * (z + 0.044715 * z * z * z)))
        return p + z * p * (1 - p) * u * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def _plain_gated(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    g, u = x @ s["wg"].float().T, x @ s["wu"].float().T
    if c["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    h = (_act(c["act"], g) * u).to(dt)
    return {"h": h, "g": g.to(dt) if c["keep"] else None, "u": u.to(dt) if c["keep"] else None}


def _plain_gated_grad(s):
    c, dt = s["case"], s["x"].dtype
    dh, g, u, x = s["dh"].float(), s["g"].float(), s["u"].float(), s["x"].float()
    du = dh * _act(c["act"], g)
    dg = dh * u * _slope(c["act"], g)
    out = {"dx": dg @ s["wg"].float() + du @ s["wu"].float(), "dwg": dg.T @ x, "dwu": du.T @ x}
    out.update(dbg=dg.sum(0) if c["bias"] else None, dbu=du.sum(0) if c["bias"] else None)
    return {k: None if v is None else v.to(dt) for k, v in out.items()}


def _plain_distill(s):
    c = s["case"]
    alpha, tau = c["alpha"], c["tau"]
    x, w = s["logits"].float(), s["weights"]
    top = x.max(1, keepdim=True).values
    x = x - top
    loss, grad = torch.zeros(c["t"], device=DEV), torch.zeros_like(x)
    if alpha < 1:
        e = torch.exp(x)
        total = e.sum(1, keepdim=True)
        there = s["targets"] >= 0
        at = s["targets"].long().clamp(min=0)[:, None]
        loss = loss + torch.where(there, (1 - alpha) * (total.log() - x.gather(1, at))[:, 0], 0.0)
        grad = grad + torch.where(there[:, None], (1 - alpha) * (e / total), 0.0)
        grad.scatter_add_(1, at, torch.where(there, alpha - 1.0, 0.0)[:, None])
    if alpha > 0:
        z = s["teacher"].float() / tau
        p = torch.exp(z - z.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        e = torch.exp(x / tau)
        total = e.sum(1, keepdim=True)
        index = s["index"].long()
        terms = p * (p.log() - (x.gather(1, index) / tau - total.log()))
        loss = loss + alpha * tau * tau * torch.where(p > 0, terms, 0.0).sum(1)
        grad = grad + alpha * tau * (e / total)
        grad.scatter_add_(1, index, -alpha * tau * p)
    on = w != 0
    grad = torch.where(on[:, None], grad * (GRAD_SCALE * w)[:, None], 0.0)
    return {"loss": torch.where(on, loss * w, 0.0), "dlogits": grad.to(s["logits"].dtype)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------


def exact(c, seed):
    s = _inputs(c, seed)
    f, op = torch.float64, c["op"]
    d = {k: v.to(f) for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "embed":
        padded = torch.cat((d["table"] * SCALE, torch.zeros((1, c["d"]), dtype=f, device=DEV)))
        return torch.index_select(padded, 0, torch.where(s["ids"] < 0, c["v"], s["ids"]).long())
    if op == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        ids, rows = s["ids"][order].long(), d["dy"][order]
        keep = ids >= 0
        out = torch.zeros((c["v"], c["d"]), dtype=f, device=DEV)
        out.index_add_(0, ids[keep], rows[keep])
        return out * SCALE + (d["dtable"] if c["add"] else 0)
    if op == "norm":
        var, mean = torch.var_mean(d["x"], dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(d["b"], (d["x"] - mean[:, None]) * rstd[:, None], d["w"]), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        n, r = c["d"], d["rstd"][:, None]
        hat = (d["x"] - d["mean"][:, None]) * r
        a = d["dy"] * d["w"]
        dx = (a * n - a.sum(1, keepdim=True) - hat * torch.einsum("td,td->t", a, hat)[:, None]) * (r / n)
        if c["residual"]:
            dx += d["res"]
        return {"dx": dx, "dw": torch.einsum("td,td->d", d["dy"], hat), "db": d["dy"].sum(0)}
    if op == "distill":
        live = (s["weights"] != 0).to(f)
        w = d["weights"]
        loss = torch.zeros(c["t"], dtype=f, device=DEV)
        grad = torch.zeros((c["t"], c["v"]), dtype=f, device=DEV)
        if c["alpha"] < 1:
            lq = torch.log_softmax(d["logits"], 1)
            at = s["targets"].long()
            on = torch.nonzero(at >= 0)[:, 0]
            loss[on] -= (1 - c["alpha"]) * lq[on, at[on]]
            part = lq[on].exp_()
            part[torch.arange(len(on), device=DEV), at[on]] -= 1
            grad[on] += part * (1 - c["alpha"])
            del lq, part
        if c["alpha"] > 0:
            tau = c["tau"]
            lp = torch.log_softmax(d["teacher"] / tau, 1)
            lq = torch.log_softmax(d["logits"] / tau, 1)
            at = s["index"].long()
            loss += c["alpha"] * tau**2 * (lp.exp() * (lp - torch.take_along_dim(lq, at, 1))).sum(1)
            q = lq.exp_()
            q.scatter_add_(1, at, -lp.exp())
            grad += q * (c["alpha"] * tau)
        return {"loss": loss * w, "dlogits": grad * (live * w * GRAD_SCALE)[:, None]}
    act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[c["act"]]
    if op == "gated":
        zero = torch.zeros(c["n"], dtype=f, device=DEV)
        g, u = torch.addmm(d.get("bg", zero), d["x"], d["wg"].T), torch.addmm(d.get("bu", zero), d["x"], d["wu"].T)
        return {"h": act(g) * u, "g": g if c["keep"] else None, "u": u if c["keep"] else None}
    g = d["g"].detach().requires_grad_()
    with torch.enable_grad():
        a = act(g)
        (slope,) = torch.autograd.grad(a.sum(), g)
    dg, du = d["dh"] * d["u"] * slope, d["dh"] * a.detach()
    return {"dx": torch.addmm(du @ d["wu"], dg, d["wg"]), "dwg": dg.T @ d["x"], "dwu": du.T @ d["x"],
            "dbg": dg.sum(0) if c["bias"] else None, "dbu": du.sum(0) if c["bias"] else None}
