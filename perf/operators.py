"""The network operators of a per-Gaussian attribute decoder: layer norm, the
linear layer with its epilogue, and the linear layer whose weights go by
group (one decoder head per block of the scene), each forward and backward.

    norm      y = gamma (x - mean) rstd + beta over the last axis
    linear    z = x w^T + bias;  y = act(z) + residual
    grouped   the same with w[e], bias[e] for the rows offsets[e] ..
              offsets[e + 1] (ragged, some empty)

`listed()` names the cases, `draw()` makes more of the same ranges,
`prepare()` the inputs, `run()` one pass, either in elementary torch
operations in 32 bits (``own`` false) or through the library (``own`` true),
`exact()` the same results in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5

# what a drawn case may cost at most (all below the largest listed ones)
MAX_FLOPS = 5.0e11
MAX_ELEMENTS = 4.0e8
MAX_WEIGHTS = 1.6e7


def _norm(way, rows, width, dtype, **kw):
    return dict(op="norm_" + way, rows=rows, width=width, dtype=dtype, **kw)


def _linear(way, rows, inner, outer, dtype, act="none", groups=0, **kw):
    return dict(op=("grouped_" if groups else "linear_") + way, rows=rows, inner=inner, outer=outer, dtype=dtype,
                act=act, groups=groups, **kw)


def listed():
    return [
        # one Gaussian's features: what a call costs
        dict(name="norm_one_row", **_norm("fwd", 1, 256, "bf16")),
        # the features of the mid scene's million Gaussians
        dict(name="norm_mid", **_norm("fwd", 1_000_000, 256, "bf16")),
        # rows that no vector width divides, fp32 as the parameter planes,
        # with the residual branch's gradient added
        dict(name="norm_bwd_odd", **_norm("bwd", 100_003, 515, "fp32", residual=True)),
        dict(name="norm_bwd_mid", **_norm("bwd", 1_000_000, 256, "bf16", residual=False)),
        # one row through a wide layer: the weights' bytes
        dict(name="linear_one_row", **_linear("fwd", 1, 4096, 4096, "bf16", "silu", residual=False, save=False)),
        # the decoder's first layer over the mid scene, in training (the
        # value before the activation is kept for the backward pass)
        dict(name="linear_mid", **_linear("fwd", 1_000_000, 64, 256, "bf16", "gelu", residual=False, save=True)),
        # matrix-rate bound, with every part of the epilogue
        dict(name="linear_large", **_linear("fwd", 16_384, 4096, 4096, "fp16", "relu", residual=True, save=False)),
        # the head onto the 59 parameters of a Gaussian, fp32, odd sizes
        dict(name="linear_bwd_odd", **_linear("bwd", 50_001, 251, 59, "fp32", "none")),
        # a hidden layer of the decoder over the mid scene
        dict(name="linear_bwd_mid", **_linear("bwd", 1_000_000, 256, 256, "bf16", "gelu")),
        # a handful of rows over many heads: most heads see none
        dict(name="grouped_few", **_linear("fwd", 32, 1024, 2048, "bf16", "silu", 64, residual=False, save=False)),
        # per-block heads over a large visible set
        dict(name="grouped_mid", **_linear("fwd", 400_000, 256, 512, "bf16", "gelu", 16, residual=False, save=True)),
        dict(name="grouped_bwd", **_linear("bwd", 131_072, 512, 512, "fp16", "silu", 64)),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; about half of them multiples of 16."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 32:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    kind = rng.choice(["norm", "linear", "linear", "grouped", "grouped"])
    way = rng.choice(["fwd", "bwd"])
    if kind == "norm":
        width = _spread(rng, 32, 4096)
        rows = _spread(rng, 1, int(min(1_000_000, MAX_ELEMENTS / SIZE[dtype] / width)))
        return _norm(way, rows, width, dtype, **(dict(residual=rng.random() < 0.5) if way == "bwd" else {}))
    groups = rng.randint(2, 64) if kind == "grouped" else 0
    inner = _spread(rng, 32, 4096)
    outer = _spread(rng, 32, int(max(32, min(4096, MAX_WEIGHTS / (inner * max(1, groups))))))
    most = min(1_000_000, MAX_ELEMENTS / (2 * inner + 3 * outer),
               MAX_FLOPS / ((6 if way == "bwd" else 2) * inner * outer * (12 if dtype == "fp32" else 1)))
    rows = _spread(rng, 1, int(max(1, most)))
    act = rng.choice(["none", "relu", "silu", "gelu"])
    more = dict(residual=rng.random() < 0.5, save=rng.random() < 0.5) if way == "fwd" else {}
    return _linear(way, rows, inner, outer, dtype, act, groups, **more)


def _group_sizes(rows, groups, seed):
    """Ragged sizes that add up to rows: few rows fall where they fall, many
    are shared out by uneven weights with one group left empty."""
    rng = random.Random(seed * 7919 + groups)
    sizes = [0] * groups
    if rows < 16 * groups:
        for _ in range(rows):
            sizes[rng.randrange(groups)] += 1
        return sizes
    weight = [rng.uniform(0.4, 1.6) for _ in range(groups)]
    weight[rng.randrange(groups)] = 0.0
    total, left = sum(weight), rows
    for e in range(groups):
        sizes[e] = min(left, int(rows * weight[e] / total))
        left -= sizes[e]
    sizes[weight.index(max(weight))] += left
    return sizes


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(dtype)

    s = dict(case=case)
    rows = case["rows"]
    if case["op"].startswith("norm"):
        d = case["width"]
        # features whose mean and spread differ from row to row
        spread = torch.rand(rows, 1, generator=gen, device=dev) * 1.5 + 0.5
        s["x"] = (torch.randn(rows, d, generator=gen, device=dev) * spread + (spread - 1.0)).to(t)
        s["gamma"] = 1.0 + normal(d, scale=0.1, dtype=torch.float32)
        s["beta"] = normal(d, scale=0.1, dtype=torch.float32)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, d)
            s["dres"] = normal(rows, d) if case["residual"] else None
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS)
        return s
    k, n, groups = case["inner"], case["outer"], case["groups"]
    lead = (groups,) if groups else ()
    s["x"] = normal(rows, k)
    s["w"] = normal(*lead, n, k, scale=k ** -0.5)
    if groups:
        sizes = _group_sizes(rows, groups, seed)
        ends = [0]
        for v in sizes:
            ends.append(ends[-1] + v)
        s["offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
        s["longest"] = max(sizes)
    if case["op"].endswith("fwd"):
        s["bias"] = normal(*lead, n, scale=0.1, dtype=torch.float32)
        s["residual"] = normal(rows, n) if case["residual"] else None
    else:
        s["dy"] = normal(rows, n)
        s["z"] = normal(rows, n) if case["act"] != "none" else None
    return s


# --- the operators in elementary operations, 32 bits --------------------------

def _act(v, act):
    if act == "relu":
        return v.clamp_min(0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * (0.5 / math.pi) ** 0.5


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    return (c * rstd[:, None] * s["gamma"] + s["beta"]).to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["gamma"]
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _slots(s):
    """Where the rows lie once every group is filled up to the longest one:
    (group, place) of each row, and the row of each (group, place)."""
    ends, rows = s["offsets"], s["x"].shape[0]
    row = torch.arange(rows, device=ends.device)
    group = torch.searchsorted(ends[1:].contiguous(), row, right=True)
    at = ends[:-1, None] + torch.arange(s["longest"], device=ends.device)
    return group, row - ends[group], at.clamp_max(max(rows - 1, 0)), at < ends[1:, None]


def _plain_linear_fwd(s):
    case, t = s["case"], s["x"].dtype
    if case["groups"]:
        group, place, at, filled = _slots(s)
        xs = torch.where(filled[:, :, None], s["x"].float()[at], 0.0)
        z = (torch.bmm(xs, s["w"].float().transpose(1, 2)) + s["bias"][:, None, :])[group, place]
    else:
        z = s["x"].float() @ s["w"].float().t() + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(t), z.to(t)) if case["save"] else y.to(t)


def _plain_linear_bwd(s):
    case, t = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), case["act"])
    if case["groups"]:
        group, place, at, filled = _slots(s)
        gs_ = torch.where(filled[:, :, None], dz[at], 0.0)
        xs = torch.where(filled[:, :, None], s["x"].float()[at], 0.0)
        dx = torch.bmm(gs_, s["w"].float())[group, place]
        dw = torch.bmm(gs_.transpose(1, 2), xs)
        db = gs_.sum(1)
    else:
        dx, dw, db = dz @ s["w"].float(), dz.t() @ s["x"].float(), dz.sum(0)
    return dx.to(t), dw.to(t), db


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}.get(
            op, _plain_linear_fwd if op.endswith("fwd") else _plain_linear_bwd)(s)
    import differentiable_gaussian_splatting_dgs_amd as gs
    if op == "norm_fwd":
        return gs.gs_layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
    if op == "norm_bwd":
        return gs.gs_layer_norm_bwd(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], dres=s["dres"])
    act = {"none": gs.GS_ACT_NONE, "relu": gs.GS_ACT_RELU, "silu": gs.GS_ACT_SILU, "gelu": gs.GS_ACT_GELU}[case["act"]]
    if op == "linear_fwd":
        return gs.gs_linear_fwd(s["x"], s["w"], s["bias"], act, residual=s["residual"], save_z=case["save"])
    if op == "linear_bwd":
        return gs.gs_linear_bwd(s["x"], s["w"], s["dy"], s["z"], act)
    if op == "grouped_fwd":
        return gs.gs_grouped_linear_fwd(s["x"], s["w"], s["offsets"], s["bias"], act, residual=s["residual"],
                                        save_z=case["save"])
    return gs.gs_grouped_linear_bwd(s["x"], s["w"], s["offsets"], s["dy"], s["z"], act)


def work(case):
    size, rows = SIZE[case["dtype"]], case["rows"]
    if case["op"] == "norm_fwd":
        return dict(bytes=2 * rows * case["width"] * size + 8 * rows + 8 * case["width"], flops=8 * rows * case["width"])
    if case["op"] == "norm_bwd":
        planes = 4 if case["residual"] else 3
        return dict(bytes=planes * rows * case["width"] * size + 8 * rows + 12 * case["width"],
                    flops=14 * rows * case["width"])
    k, n, groups = case["inner"], case["outer"], max(1, case["groups"])
    # no more than `rows` heads can be in use
    heads = min(groups, rows)
    product = 2 * rows * k * n
    if case["op"].endswith("fwd"):
        planes = 1 + case["residual"] + case["save"]
        return dict(bytes=size * (rows * k + planes * rows * n + heads * k * n) + 4 * heads * n, flops=product)
    planes = 2 if case["act"] != "none" else 1
    return dict(bytes=size * (2 * rows * k + planes * rows * n + (heads + groups) * k * n) + 4 * groups * n,
                flops=2 * product)


# --- the definitions in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    x = s["x"].to(f64)
    if case["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / (var + EPS).sqrt()
        return [s["gamma"].to(f64) * ((x - mean.unsqueeze(1)) * rstd.unsqueeze(1)) + s["beta"].to(f64), mean, rstd]
    if case["op"] == "norm_bwd":
        d = case["width"]
        rstd, dy = s["rstd"].to(f64).unsqueeze(1), s["dy"].to(f64)
        unit = x.sub(s["mean"].to(f64).unsqueeze(1)).mul(rstd)
        up = dy.mul(s["gamma"].to(f64))
        dx = rstd / d * (d * up - up.sum(1, keepdim=True) - unit * torch.einsum("rd,rd->r", up, unit).unsqueeze(1))
        if case["residual"]:
            dx += s["dres"].to(f64)
        return [dx, torch.einsum("rd,rd->d", dy, unit), torch.ones(1, case["rows"], dtype=f64, device=x.device).mm(dy)[0]]
    groups = case["groups"]
    ends = s["offsets"].tolist() if groups else [0, case["rows"]]
    w = s["w"].to(f64).reshape(len(ends) - 1, case["outer"], case["inner"])
    spans = list(zip(ends[:-1], ends[1:]))
    half = math.sqrt(0.5)
    if case["op"].endswith("fwd"):
        bias = s["bias"].to(f64).reshape(len(spans), -1)
        z = torch.cat([torch.addmm(bias[e], x[a:b], w[e].t()) for e, (a, b) in enumerate(spans)])
        y = {"none": lambda v: v, "relu": lambda v: torch.where(v > 0, v, torch.zeros_like(v)),
             "silu": lambda v: v * torch.sigmoid(v), "gelu": lambda v: 0.5 * v * torch.erfc(-v * half)}[case["act"]](z)
        if case["residual"]:
            y = y + s["residual"].to(f64)
        return [y, z] if case["save"] else y
    dz = s["dy"].to(f64)
    if case["act"] != "none":
        v = s["z"].to(f64)
        if case["act"] == "relu":
            dz = torch.where(v > 0, dz, torch.zeros_like(dz))
        elif case["act"] == "silu":
            p = torch.sigmoid(v)
            dz = dz * (p + v * p * torch.sigmoid(-v))
        else:
            dz = dz * (0.5 * torch.erfc(-v * half) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi))
    dx = torch.cat([dz[a:b].mm(w[e]) for e, (a, b) in enumerate(spans)])
    dw = torch.stack([dz[a:b].t().mm(x[a:b]) for a, b in spans])
    db = torch.stack([dz[a:b].sum(0) for a, b in spans])
    return [dx, dw, db] if groups else [dx, dw[0], db[0]]
