"""Cases of the framework's training operators: the AdamW step over many tensors (states in 32
or in 8 bits), the global gradient norm with its clipping factor, and the linear layer with bias,
activation and residual, forward and backward.

``run`` computes a case either in plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where ``own`` is true, by the framework's calls.  ``exact`` computes it in 64 bits.

Tensors of one optimizer case live in flat arenas, one per stream (gradients, master, moments,
parameters), as a training program that allocates once keeps them; in a "packed" arena they follow
each other directly, in a "padded" one each starts on a multiple of 256 elements.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 256  # elements that share one scale of an 8-bit state
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETA1, BETA2, EPS, STEP = 1e-3, 0.9, 0.999, 1e-8, 100
DECAY = 0.1  # on matrices; vectors (biases, norms) have none


def listed():
    return [
        # one small two-layer MLP (what an example or a probe trains): latency of a call
        dict(name="adamw32-small", op="adamw", bits=32, d=64, layers=1, tail=0, ranks=2, grad="fp16", param="fp16", layout="packed"),
        # four blocks of the 1.3e9-parameter model, eight ranks' bf16 gradients
        dict(name="adamw32-4blocks-p8", op="adamw", bits=32, d=2048, layers=4, tail=0, ranks=8, grad="bf16", param="bf16", layout="padded"),
        # the whole 1.3e9-parameter model, 24 blocks and an embedding, one gradient
        dict(name="adamw32-1p3b", op="adamw", bits=32, d=2048, layers=24, tail=91401472, ranks=1, grad="fp16", param="fp16", layout="packed"),
        # odd widths: every matrix and vector ends inside a block of scales
        dict(name="adamw8-odd", op="adamw", bits=8, d=331, layers=3, tail=10007, ranks=1, grad="fp32", param="fp16", layout="padded"),
        # the whole model with 8-bit states
        dict(name="adamw8-1p3b", op="adamw", bits=8, d=2048, layers=24, tail=91401472, ranks=1, grad="bf16", param="bf16", layout="padded"),
        # clipping of a small model: latency
        dict(name="norm-small", op="norm", d=64, layers=1, tail=0, ranks=2, grad="fp16", layout="packed"),
        # clipping of eight ranks' gradients of six blocks
        dict(name="norm-6blocks-p8", op="norm", d=2048, layers=6, tail=0, ranks=8, grad="fp16", layout="packed"),
        # a few tokens through the up-projection of a d = 2048 block (generation, tiny batches)
        dict(name="linear-4tokens", op="linear", t=4, k=2048, n=8192, act="gelu", residual=False, keep_z=False, type="bf16", pad=0),
        # the down-projection of a training batch, with the residual
        dict(name="linear-down-16k", op="linear", t=16384, k=8192, n=2048, act="none", residual=True, keep_z=False, type="fp16", pad=0),
        # odd sizes and rows off the 16-byte boundary
        dict(name="linear-odd", op="linear", t=1009, k=1001, n=1543, act="silu", residual=True, keep_z=True, type="bf16", pad=3),
        # the gradients of the up-projection of a training batch
        dict(name="backward-up-8k", op="backward", t=8192, k=2048, n=8192, act="gelu", type="bf16", pad=0),
        # gradients of odd sizes, few rows
        dict(name="backward-odd", op="backward", t=509, k=777, n=1190, act="relu", type="fp16", pad=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm", "linear", "backward"])
    if op in ("adamw", "norm"):
        d = _log(rng, 40, 2300)
        layers = max(1, min(24, int(4e8 / (12 * d * d)), _log(rng, 1, 24)))
        d += d in (768, 1024)
        c = dict(op=op, d=d, layers=layers, tail=rng.choice([0, _log(rng, 100, 5000000)]), ranks=rng.choice([1, 1, 2, 3, 4, 8]),
                 grad=rng.choice(["fp16", "bf16", "fp32"]), layout=rng.choice(["packed", "padded"]))
        if op == "adamw":
            c.update(bits=rng.choice([8, 32]), param=rng.choice(["fp16", "bf16"]))
            if c["bits"] == 8:
                c["layout"] = "padded"
        return c
    t, k, n = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 8192)
    if rng.random() < 0.5:  # widths as models have them
        k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
    t = max(1, min(t, int((5.4e11 if op == "linear" else 2.7e11) / (2 * k * n))))
    t, k, n = (v - (v == 3072) for v in (t, k, n))
    c = dict(op=op, t=t, k=k, n=n, act=rng.choice(["none", "relu", "gelu", "silu"]), type=rng.choice(["fp16", "bf16"]), pad=rng.choice([0, 0, 1, 8]))
    if op == "linear":
        c.update(residual=rng.random() < 0.5, keep_z=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------------------------
# shapes
# ---------------------------------------------------------------------------------------------


def _sizes(c):
    """(elements, is a matrix) of each tensor: blocks of two norms (weight and bias each), fused qkv, output projection and
    the two MLP projections with their biases; then one table of `tail` elements."""
    d = c["d"]
    block = [(d, 0), (d, 0), (3 * d * d, 1), (3 * d, 0), (d * d, 1), (d, 0), (d, 0), (d, 0), (4 * d * d, 1), (4 * d, 0), (4 * d * d, 1), (d, 0)]
    return block * c["layers"] + ([(c["tail"], 1)] if c["tail"] else [])


def _layout(c):
    """(elements, offset, decay) of each tensor, and the arena's length."""
    q = BLOCK if c["layout"] == "padded" else 1
    at, out = 0, []
    for n, matrix in _sizes(c):
        out.append((n, at, DECAY if matrix else 0.0))
        at += -(-n // q) * q
    return out, at


def _elems(c):
    return sum(n for n, _ in _sizes(c))


def work(c):
    if c["op"] in ("adamw", "norm"):
        n, g = _elems(c), 4 if c["grad"] == "fp32" else 2
        if c["op"] == "norm":
            return {"bytes": n * g * c["ranks"], "flops": n * (c["ranks"] + 3)}
        state = 24 if c["bits"] == 32 else 12 + 16 / BLOCK
        return {"bytes": n * (g * c["ranks"] + state + 2), "flops": n * (c["ranks"] + 15)}
    t, k, n = c["t"], c["k"], c["n"]
    if c["op"] == "linear":
        moved = t * k + n * k + n + t * n * (1 + c["residual"] + c["keep_z"])
        return {"bytes": 2 * moved, "flops": 2 * t * k * n}
    moved = t * n * (1 + (c["act"] != "none")) + t * k + n * k + t * k + n * k + n
    return {"bytes": 2 * moved, "flops": 4 * t * k * n}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = _prepare_optimizer(c, gen, seed) if c["op"] in ("adamw", "norm") else _prepare_linear(c, gen)
    s["case"] = c
    if own:
        _attach(s)
    return s


def _zero_gaps(a, tensors):
    ends = [at for _, at, _ in tensors[1:]] + [a.shape[-1]]
    for (n, at, _), end in zip(tensors, ends):
        if at + n < end:
            a[..., at + n : end] = 0


def _prepare_optimizer(c, gen, seed):
    tensors, total = _layout(c)
    stride = -(-total // 8) * 8
    grads = torch.empty((c["ranks"], stride), dtype=TYPES[c["grad"]], device=DEV)
    for r in range(c["ranks"]):
        grads[r] = torch.randn(stride, generator=gen, device=DEV) * 1e-3
    _zero_gaps(grads, tensors)
    grads[:, total:] = 0
    s = {"tensors": tensors, "total": total, "grads": grads, "stats": torch.zeros(3, device=DEV)}
    if c["op"] == "norm":
        return s
    # clipping's answer for these gradients, as the step gets it: norm, factor, finite
    s["stats"].copy_(torch.tensor([2.5, 0.4, 1.0]))
    master = torch.randn(total, generator=gen, device=DEV) * 0.02
    m = torch.randn(total, generator=gen, device=DEV) * 3e-4
    v = (torch.rand(total, generator=gen, device=DEV) + 0.2) * 1e-6
    for a in (master, m, v):
        _zero_gaps(a, tensors)
    s.update(master=master, param=master.to(TYPES[c["param"]]), seed=seed & 0x7FFFFFFF)
    if c["bits"] == 32:
        s.update(m=m, v=v)
        return s
    for name, a in (("m", m), ("v", v.sqrt_())):
        a = a.view(-1, BLOCK)
        scale = a.abs().amax(1) * (1 / 448)
        s[name] = (a / scale[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(-1)
        s[name + "_scale"] = scale
    return s


def _rows(t, width, pad, dtype, gen, scale):
    """[t, width] values in rows of width + pad elements."""
    return (torch.randn((t, width + pad), generator=gen, device=DEV) * scale).to(dtype)[:, :width]


def _prepare_linear(c, gen):
    t, k, n, dt, pad = c["t"], c["k"], c["n"], TYPES[c["type"]], c["pad"]
    s = {"x": _rows(t, k, pad, dt, gen, 1.0), "w": _rows(n, k, pad, dt, gen, 1 / math.sqrt(k)), "y": None, "z": None, "res": None}
    if c["op"] == "linear":
        s["bias"] = (torch.randn(n, generator=gen, device=DEV) * 0.1).to(dt)
        s["y"] = torch.empty((t, n + pad), dtype=dt, device=DEV)[:, :n]
        if c["keep_z"]:
            s["z"] = torch.empty((t, n + pad), dtype=dt, device=DEV)[:, :n]
        if c["residual"]:
            s["res"] = _rows(t, n, pad, dt, gen, 1.0)
        return s
    s["dy"] = _rows(t, n, pad, dt, gen, 0.1)
    if c["act"] != "none":
        s["z"] = _rows(t, n, pad, dt, gen, 1.0)
    s["dx"] = torch.empty((t, k + pad), dtype=dt, device=DEV)[:, :k]
    s["dw"] = torch.empty((n, k), dtype=dt, device=DEV)
    s["db"] = torch.empty(n, dtype=dt, device=DEV)
    return s


def _attach(s):
    """The plan or workspace that a program keeps for the framework's calls."""
    import zero_sharded_mixed_shard_gb300 as z

    c = s["case"]
    s["z_"] = z
    types = {"fp16": z.TYPE_FP16, "bf16": z.TYPE_BF16, "fp32": z.TYPE_FP32}
    if c["op"] in ("adamw", "norm"):
        rows, blocks = [], 0
        stride = s["grads"].shape[1]
        for n, at, decay in s["tensors"]:
            row = dict(grad=s["grads"][0, at:], rank_stride=stride, n=n, weight_decay=decay)
            if c["op"] == "adamw":
                row.update(master=s["master"][at:], m=s["m"][at:], v=s["v"][at:], param=s["param"][at:])
                if c["bits"] == 8:
                    row.update(m_scale=s["m_scale"][at // BLOCK :], v_scale=s["v_scale"][at // BLOCK :])
            rows.append(row)
        if c["op"] == "norm":
            s["plan"] = z.zero_grad_plan(rows, c["ranks"], types[c["grad"]])
        else:
            s["plan"] = z.zero_adamw_plan(rows, c["ranks"], types[c["grad"]], types[c["param"]], c["bits"])
        return
    s["act"] = {"none": z.ACT_NONE, "relu": z.ACT_RELU, "gelu": z.ACT_GELU, "silu": z.ACT_SILU}[c["act"]]
    s["type"] = types[c["type"]]
    aligned = all(t is None or (t.data_ptr() % 16 == 0 and t.stride(0) % 8 == 0) for t in (s["x"], s["w"], s.get("dy"), s.get("z"), s.get("dx"), s.get("dw")))
    need = z.zero_linear_workspace(c["t"], c["k"], c["n"], s["act"], c["op"] == "backward", aligned)
    s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"adamw": _own_adamw, "norm": _own_norm, "linear": _own_linear, "backward": _own_backward}[op](s)
    return {"adamw": _plain_adamw, "norm": _plain_norm, "linear": _plain_linear, "backward": _plain_backward}[op](s)


def _own_adamw(s):
    s["z_"].zero_adamw_step(s["plan"], s["stats"], STEP, LR, BETA1, BETA2, EPS, s["seed"])
    return {k: s[k] for k in ("master", "param", "m", "v", "m_scale", "v_scale") if k in s}


def _own_norm(s):
    s["z_"].zero_grad_norm(s["plan"], 1.0, 1.0, s["stats"])
    return s["stats"]


def _own_linear(s):
    c, x, w, y, z, res = s["case"], s["x"], s["w"], s["y"], s["z"], s["res"]
    s["z_"].zero_linear_forward(x, x.stride(0), w, w.stride(0), s["bias"], res, res.stride(0) if res is not None else 0, y, y.stride(0),
                                z, z.stride(0) if z is not None else 0, c["t"], c["k"], c["n"], s["act"], s["type"], s["ws"], s["ws"].numel())
    return {"y": y, "z": z}


def _own_backward(s):
    c, x, w, dy, z, dx, dw = s["case"], s["x"], s["w"], s["dy"], s["z"], s["dx"], s["dw"]
    s["z_"].zero_linear_backward(dy, dy.stride(0), z, z.stride(0) if z is not None else 0, x, x.stride(0), w, w.stride(0), dx, dx.stride(0),
                                 dw, dw.stride(0), s["db"], c["t"], c["k"], c["n"], s["act"], s["type"], s["ws"], s["ws"].numel())
    return {"dx": dx, "dw": dw, "db": s["db"]}


def _f32(x):
    return float(np.float32(x))


def _mean(s):
    """The ranks' mean gradient, summed in rank order."""
    g = s["grads"][:, : s["total"]]
    total = g[0].float()
    for r in range(1, g.shape[0]):
        total = total + g[r].float()
    return total if g.shape[0] == 1 else total / torch.full((), g.shape[0], dtype=torch.float32, device=DEV)


def _spread(s, values, dtype):
    """One value of each tensor, for every element of the arena."""
    ends = [at for _, at, _ in s["tensors"][1:]] + [s["total"]]
    counts = torch.tensor([end - at for (_, at, _), end in zip(s["tensors"], ends)], device=DEV)
    return torch.repeat_interleave(torch.tensor(values, dtype=dtype, device=DEV), counts, output_size=s["total"])


def _mix(h):
    """MurmurHash3's 32-bit finaliser (A. Appleby), on 64-bit integers."""
    low = 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & low
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & low
    return h ^ (h >> 16)


def _random16(s):
    """Sixteen random bits for each element of the arena: of its pair of elements in its tensor and the call's seed."""
    base = _mix(torch.tensor(s["seed"], device=DEV))
    keys = _mix((base + 0x9E3779B9 * torch.arange(1, len(s["tensors"]) + 1, device=DEV)) & 0xFFFFFFFF)
    ends = [at for _, at, _ in s["tensors"][1:]] + [s["total"]]
    counts = torch.tensor([(end - at) // 2 for (_, at, _), end in zip(s["tensors"], ends)], device=DEV)
    first = torch.tensor([at // 2 for _, at, _ in s["tensors"]], device=DEV)
    size = s["total"] // 2
    pair = torch.arange(size, device=DEV) + torch.repeat_interleave(keys - first, counts, output_size=size)
    h = _mix(pair & 0xFFFFFFFF)
    return torch.stack((h & 0xFFFF, h >> 16), 1).view(-1).int()


def _plain_adamw(s):
    c = s["case"]
    b1, b2, lr, decay = _f32(BETA1), _f32(BETA2), _f32(LR), _f32(_f32(LR) * _f32(DECAY))
    o1, o2 = _f32(np.float32(1) - np.float32(b1)), _f32(np.float32(1) - np.float32(b2))
    r1, c2 = _f32(1 / (1 - b1**STEP)), _f32(1 / math.sqrt(1 - b2**STEP))
    go = s["stats"][2] > 0
    g = _mean(s) * s["stats"][1]
    if c["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        root = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1)
        v = root * root
    else:
        m, v = s["m"], s["v"]
    m = m * b1 + g * o1
    v = v * b2 + (g * g) * o2
    root = v.sqrt()
    w = s["master"]
    w = w - _spread(s, [decay if d else 0.0 for _, _, d in s["tensors"]], torch.float32) * w
    w = w - ((m * r1) / (root * c2 + _f32(EPS))) * lr
    new = {"master": w, "param": w.to(TYPES[c["param"]])}
    if c["bits"] == 32:
        new.update(m=m, v=v)
    else:
        top = torch.tensor(448.0)
        m, root = m.view(-1, BLOCK), root.view(-1, BLOCK)
        high_m, high_r = m.abs().amax(1, keepdim=True), root.amax(1, keepdim=True)
        inv_m = torch.where(high_m < 2.0**-96, 0.0, top / high_m)
        inv_r = torch.where(high_r < 2.0**-96, 0.0, top / high_r)
        new["m"] = (m * inv_m).to(torch.float8_e4m3fn).view(-1)
        # stochastic rounding: the value scaled so that a code is the top bits of its binary32 form, plus random low bits
        y = (root * inv_r).view(-1)
        bits = ((y * 2.0**-120).view(torch.int32) + (_random16(s) << 4)) >> 20
        bits = torch.where(y > 0, bits.clamp(1, 0x7E), 0)
        new["v"] = bits.to(torch.uint8).view(torch.float8_e4m3fn)
        new["m_scale"] = torch.where(high_m < 2.0**-96, 0.0, high_m * _f32(1 / 448)).view(-1)
        new["v_scale"] = torch.where(high_r < 2.0**-96, 0.0, high_r * _f32(1 / 448)).view(-1)
    byte = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    for k, t in new.items():
        byte(s[k]).copy_(torch.where(go, byte(t), byte(s[k])))
    return {k: s[k] for k in ("master", "param", "m", "v", "m_scale", "v_scale") if k in s}


def _plain_norm(s):
    norm = _mean(s).square().sum().sqrt()
    finite = torch.isfinite(norm)
    factor = (1.0 / (norm + 1e-6)).clamp(max=1.0)
    return torch.stack((norm, torch.where(finite, factor, 0.0), finite.float()))


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


def _plain_linear(s):
    c = s["case"]
    dt = TYPES[c["type"]]
    z = s["x"].float() @ s["w"].float().T + s["bias"].float()
    y = _act(c["act"], z)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(dt), "z": z.to(dt) if c["keep_z"] else None}


def _plain_backward(s):
    c = s["case"]
    dt = TYPES[c["type"]]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _slope(c["act"], s["z"].float())
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.T @ s["x"].float()).to(dt), "db": dz.sum(0).to(dt)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------


def exact(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    f = torch.float64
    if c["op"] in ("linear", "backward"):
        s = _prepare_linear(c, gen)
        x, w = s["x"].to(f), s["w"].to(f)
        if c["op"] == "linear":
            z = torch.addmm(s["bias"].to(f), x, w.T)
            y = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: torch.nn.functional.silu(z),
                 "gelu": lambda: torch.nn.functional.gelu(z, approximate="tanh")}[c["act"]]()
            return {"y": y if s["res"] is None else y + s["res"].to(f), "z": z if c["keep_z"] else None}
        dz = s["dy"].to(f)
        if c["act"] != "none":
            z = s["z"].to(f)
            if c["act"] == "relu":
                dz = torch.where(z > 0, dz, torch.zeros_like(dz))
            elif c["act"] == "silu":
                dz = dz * torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
            else:
                k = math.sqrt(2 / math.pi)
                th = torch.tanh(k * (z + 0.044715 * z**3))
                dz = dz * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * k * (1 + 3 * 0.044715 * z * z))
        return {"dx": dz @ w, "dw": dz.T @ x, "db": dz.sum(0)}
    s = _prepare_optimizer(c, gen, seed)
    total = s["total"]
    g = torch.zeros(total, dtype=f, device=DEV)
    for row in s["grads"]:
        g += row[:total].to(f)
    g /= c["ranks"]
    if c["op"] == "norm":
        norm = torch.linalg.vector_norm(g)
        return torch.stack((norm, torch.clamp(1 / (norm + 1e-6), max=1.0), torch.ones_like(norm)))
    g *= 0.4
    if c["bits"] == 32:
        m, v = s["m"].to(f), s["v"].to(f)
    else:
        m = (s["m"].to(f).view(-1, BLOCK) * s["m_scale"].to(f)[:, None]).view(-1)
        v = (s["v"].to(f).view(-1, BLOCK) * s["v_scale"].to(f)[:, None]).view(-1).square_()
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    del g
    w = s["master"].to(f)
    step = m / (1 - BETA1**STEP) / ((v / (1 - BETA2**STEP)).sqrt_() + EPS)
    for n, at, decay in s["tensors"]:
        w[at : at + n] *= 1 - LR * decay
    w.sub_(step, alpha=LR)
    out = {"master": w, "param": w}
    if c["bits"] == 32:
        return dict(out, m=m, v=v)
    # a code stands for a rounding of the moment over its block's scale; the moment itself, unrounded, is what it is held to
    for name, a in (("m", m), ("v", v.sqrt_())):
        a = a.view(-1, BLOCK)
        scale = a.abs().amax(1) / 448
        out[name + "_scale"] = scale
        out[name] = (a / scale[:, None].clamp(min=1e-300)).view(-1)
    return out
