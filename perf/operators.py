"""What the training and serving products of the layer are measured on.

Three operators, each in both directions:

* ``linear``: y = act(x W^T + b) + residual, and its gradients (a dense projection of the model);
* ``grouped``: the experts' products, rows grouped by expert with ragged sizes, y_r = W_e x_r + b_e for
  the rows r of expert e, and its gradients;
* ``swiglu``: h = SiLU(min(g, L)) * clamp(u, -L, L) between an expert's products, and its gradients.

``own`` chooses the plain form in torch operations or the package's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token through a 4096 -> 1280 projection with everything in the epilogue: pure
        # latency and weight streaming
        dict(name="linear_token", op="linear", back=False, rows=1, k=4096, n=1280, act="silu",
             residual=True, keep_z=False, out="bf16"),
        # a decode batch through the dense layers' 11264 -> 4096 down projection, residual added
        dict(name="linear_decode", op="linear", back=False, rows=64, k=11264, n=4096, act="none",
             residual=True, keep_z=False, out="bf16"),
        # a ragged prompt through odd widths (no tile size divides any of them) into fp32 logits
        dict(name="linear_odd", op="linear", back=False, rows=777, k=1288, n=2056, act="none",
             residual=False, keep_z=False, out="f32"),
        # the training forward of a wide GELU projection; z is kept for the backward pass
        dict(name="linear_train", op="linear", back=False, rows=8192, k=4096, n=11264, act="gelu",
             residual=False, keep_z=True, out="bf16"),
        # its backward pass on a smaller batch
        dict(name="linear_train_back", op="linear", back=True, rows=4096, k=4096, n=11264,
             act="gelu", out="bf16"),
        # the backward pass of a plain projection, weight gradient in fp32, an odd batch
        dict(name="linear_back_f32", op="linear", back=True, rows=2049, k=4096, n=1280, act="none",
             out="f32"),
        # a decode batch's gate product: 64 tokens on 8 of 288 experts each, few rows per expert
        dict(name="grouped_decode", op="grouped", back=False, rows=512, groups=288, k=4096, n=1280,
             per_token=8, skew=1.0, bias=False, out="bf16"),
        # a prompt's gate product: 8192 tokens on 8 of 288 experts
        dict(name="grouped_prefill", op="grouped", back=False, rows=65536, groups=288, k=4096,
             n=1280, per_token=8, skew=0.5, bias=False, out="bf16"),
        # a few tokens on small experts, odd sizes, with biases: latency
        dict(name="grouped_small", op="grouped", back=False, rows=77, groups=16, k=264, n=200,
             per_token=1, skew=0.5, bias=True, out="bf16"),
        # the training backward of 48 experts at top 3: input, weight and bias gradients
        dict(name="grouped_back", op="grouped", back=True, rows=24576, groups=48, k=4096, n=1280,
             per_token=3, skew=0.5, bias=True, out="f32"),
        # the activation of a prompt's routed rows, clamped as in the model's last layers
        dict(name="swiglu_prefill", op="swiglu", back=False, rows=65536, n=1280, limit=7.0),
        # its backward pass in training, h recomputed on the way
        dict(name="swiglu_back", op="swiglu", back=True, rows=24576, n=1280, limit=7.0),
    ]


def _size(rng, low, high, step):
    """A multiple of `step` between low and high, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(high, max(low, round(v / step) * step)))


def draw(rng):
    while True:
        op = rng.choice(("linear", "linear", "grouped", "grouped", "swiglu"))
        back = rng.random() < 0.5
        rows = _size(rng, 1 if not back else 16, 65536, 1)
        k, n = _size(rng, 64, 11264, 8), _size(rng, 64, 11264, 8)
        if op == "linear":
            act = rng.choice(ACTS)
            c = dict(op=op, back=back, rows=rows, k=k, n=n, act=act)
            if back:  # a gradient through an activation leaves in bf16
                c.update(out=rng.choice(("bf16", "f32")) if act == "none" else "bf16")
            else:
                c.update(residual=rng.random() < 0.5, keep_z=act != "none" and rng.random() < 0.5,
                         out=rng.choice(("bf16", "f32")))
        elif op == "grouped":
            c = dict(op=op, back=back, rows=rows, groups=_size(rng, 2, 288, 1), k=k, n=n,
                     per_token=rng.choice((1, 2, 3, 4, 8)), skew=rng.choice((0.0, 0.5, 1.0)),
                     bias=rng.random() < 0.5, out=rng.choice(("bf16", "f32")))
            if c["groups"] * k * n > 1_600_000_000:
                continue
        else:
            c = dict(op=op, back=back, rows=rows, n=n, limit=rng.choice((0.0, 7.0)))
        w = work(c)
        if w["flops"] <= 7.6e11 and w["bytes"] <= 3.5e9:
            return c


def _group_sizes(case):
    """Rows of each expert, busiest first: proportional to rank ** -skew."""
    e, p = case["groups"], case["rows"]
    share = [(i + 1) ** -case["skew"] for i in range(e)]
    total = sum(share)
    sizes = [int(p * s / total) for s in share]
    for i in range(p - sum(sizes)):
        sizes[i % e] += 1
    return sizes


def work(case):
    if case["op"] == "swiglu":
        v = case["rows"] * case["n"]
        return {"bytes": v * 2 * (6 if case["back"] else 3), "flops": v * (20 if case["back"] else 8)}
    p, k, n = case["rows"], case["k"], case["n"]
    f32 = 4 if case["out"] == "f32" else 2
    if case["op"] == "linear":
        if not case["back"]:
            return {"bytes": 2 * p * k + 2 * n * k + 4 * n + f32 * p * n
                    + 2 * p * n * (case["residual"] + case["keep_z"]), "flops": 2 * p * n * k}
        z = 2 if case["act"] != "none" else 0  # z read, dz written
        return {"bytes": 2 * p * n * (1 + z) + 2 * (2 * p * k + n * k) + f32 * n * k + 4 * n,
                "flops": 4 * p * n * k}
    active = sum(s > 0 for s in _group_sizes(case))
    tokens = -(-p // case["per_token"])
    b = 4 * n * case["bias"]
    if not case["back"]:
        return {"bytes": 2 * tokens * k + active * (2 * n * k + b) + f32 * p * n + 4 * p,
                "flops": 2 * p * n * k}
    return {"bytes": 2 * p * n + 2 * tokens * k + active * 2 * n * k + 2 * p * k
            + case["groups"] * (f32 * n * k + b) + 4 * p, "flops": 4 * p * n * k}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
        return t.mul_(scale) if scale != 1.0 else t

    s = dict(case)
    p, n = case["rows"], case["n"]
    if case["op"] == "swiglu":
        # gate and up are the halves of one product's output, as an expert's fused weight gives them
        gu = normal(p, 2 * n, scale=2.5)
        s.update(gu=gu, gate=gu[:, :n], up=gu[:, n:])
        if case["back"]:
            s.update(dh=normal(p, n, scale=0.01))
        return s
    k = case["k"]
    if case["op"] == "linear":
        s.update(x=normal(p, k), w=normal(n, k, scale=k ** -0.5))
        if case["back"]:
            s.update(dy=normal(p, n, scale=0.01), z=normal(p, n) if case["act"] != "none" else None)
        else:
            s.update(b=normal(n, scale=0.5, dtype=torch.float32),
                     r=normal(p, n) if case["residual"] else None)
        return s
    e, kt = case["groups"], case["per_token"]
    host = torch.Generator().manual_seed(seed * 104729 + 5)
    sizes = torch.tensor(_group_sizes(case))[torch.randperm(e, generator=host)]
    # the pairs (token, slot) of each expert in ascending order, as a stable sort by expert leaves them
    pairs = torch.randperm(p, generator=host)
    pairs = torch.cat([t.sort().values for t in pairs.split(sizes.tolist())])
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)])
    s.update(x=normal(-(-p // kt), k), w=normal(e, n, k, scale=k ** -0.5),
             sizes=sizes.tolist(), offsets=offsets.to(torch.int32).cuda(),
             pairs=pairs.to(torch.int32).cuda())
    if case["back"]:
        s.update(dy=normal(p, n, scale=0.01))
    else:
        s.update(b=normal(e, n, scale=0.5, dtype=torch.float32) if case["bias"] else None)
    return s


def _dtype(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def prepare(case, seed):
    s = _inputs(case, seed)
    p, n = case["rows"], case["n"]

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    # the buffers that a program keeps for the outputs
    if case["op"] == "swiglu":
        s.update(h=buf(p, n))
        if case["back"]:
            dgu = buf(p, 2 * n)
            s.update(dgu=dgu, dgate=dgu[:, :n], dup=dgu[:, n:])
    elif case["back"]:
        k = case["k"]
        e = (case["groups"],) if case["op"] == "grouped" else ()
        s.update(dx=buf(p, k), dw=buf(*e, n, k, dtype=_dtype(case)),
                 db=buf(*e, n, dtype=torch.float32) if case.get("bias", True) else None)
        if case["op"] == "linear":
            s.update(dz=buf(p, n) if case["act"] != "none" else None)
    else:
        s.update(y=buf(p, n, dtype=_dtype(case)), zout=buf(p, n) if case.get("keep_z") else None)
    return s


# ------------------------------------------------------------------ plain forms

def _act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _plain_linear(s):
    x, w = s["x"].float(), s["w"].float()
    if not s["back"]:
        z = x @ w.t() + s["b"]
        y = _act(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        out = {"y": y.to(_dtype(s))}
        if s["keep_z"]:
            out["z"] = z.to(torch.bfloat16)
        return out
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["act"])
    out = {"dx": (dz @ w).to(torch.bfloat16), "dw": (dz.t() @ x).to(_dtype(s)), "db": dz.sum(0)}
    if s["z"] is not None:
        out["dz"] = dz.to(torch.bfloat16)
    return out


def _plain_grouped(s):
    # one product per expert that has rows: ragged sizes leave torch no batched form of it
    x = s["x"][(s["pairs"] // s["per_token"]).long()].float()
    at, spans = 0, []
    for e, m in enumerate(s["sizes"]):
        spans.append((e, at, at + m))
        at += m
    if not s["back"]:
        y = torch.empty((s["rows"], s["n"]), dtype=_dtype(s), device=x.device)
        for e, i, j in spans:
            if j > i:
                v = x[i:j] @ s["w"][e].float().t()
                y[i:j] = v + s["b"][e] if s["b"] is not None else v
        return {"y": y}
    dy = s["dy"].float()
    dx = torch.empty((s["rows"], s["k"]), dtype=torch.bfloat16, device=x.device)
    dw = torch.zeros((s["groups"], s["n"], s["k"]), dtype=_dtype(s), device=x.device)
    db = torch.zeros((s["groups"], s["n"]), device=x.device)
    for e, i, j in spans:
        if j > i:
            dx[i:j] = dy[i:j] @ s["w"][e].float()
            dw[e] = dy[i:j].t() @ x[i:j]
            if s["bias"]:
                db[e] = dy[i:j].sum(0)
    return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}


def _plain_swiglu(s):
    g, u, lim = s["gate"].float(), s["up"].float(), s["limit"]
    gc, uc = (g.clamp(max=lim), u.clamp(-lim, lim)) if lim > 0 else (g, u)
    sg = torch.sigmoid(gc)
    h = gc * sg * uc
    if not s["back"]:
        return {"h": h.to(torch.bfloat16)}
    dh = s["dh"].float()
    dg, du = dh * uc * sg * (1 + gc * (1 - sg)), dh * gc * sg
    if lim > 0:
        dg, du = dg * (g <= lim), du * (u.abs() <= lim)
    return {"dgu": torch.cat([dg, du], 1).to(torch.bfloat16), "h": h.to(torch.bfloat16)}


# ------------------------------------------------------------------ the package's kernels

def _own_linear(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:  # a program makes the plan and its workspace once
        s["plan"] = moe.make_linear_config(s["rows"], s["k"], s["n"], activation=s["act"],
                                           y_dtype="bf16" if s["back"] else s["out"],
                                           dw_dtype=s["out"] if s["back"] else "f32")
        s["ws"] = moe.alloc_linear_workspace(s["plan"])
    if not s["back"]:
        moe.moe_linear_forward(s["plan"], s["x"], s["w"], s["b"], s["r"], s["y"], s["zout"], s["ws"])
        return {"y": s["y"], "z": s["zout"]} if s["keep_z"] else {"y": s["y"]}
    moe.moe_linear_backward(s["plan"], s["dy"], s["z"], s["x"], s["w"], s["dz"], s["dx"], s["dw"],
                            s["db"], s["ws"])
    out = {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    return out if s["z"] is None else {**out, "dz": s["dz"]}


def _own_grouped(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:
        s["plan"] = moe.make_grouped_config(s["rows"], s["groups"], s["k"], s["n"],
                                            x_rows=s["x"].shape[0], row_div=s["per_token"],
                                            y_dtype="bf16" if s["back"] else s["out"],
                                            dw_dtype=s["out"] if s["back"] else "f32")
        s["ws"] = moe.alloc_grouped_workspace(s["plan"])
    if not s["back"]:
        moe.moe_grouped_forward(s["plan"], s["x"], s["pairs"], s["offsets"], s["w"], s["b"], s["y"],
                                s["ws"])
        return {"y": s["y"]}
    moe.moe_grouped_backward(s["plan"], s["dy"], s["x"], s["pairs"], s["offsets"], s["w"], s["dx"],
                             s["dw"], s["db"], s["ws"])
    out = {"dx": s["dx"], "dw": s["dw"]}
    return {**out, "db": s["db"]} if s["bias"] else out


def _own_swiglu(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:
        s["plan"] = moe.make_swiglu_config(s["rows"], s["n"], ld=2 * s["n"], limit=s["limit"])
    if not s["back"]:
        moe.moe_swiglu_forward(s["plan"], s["gate"], s["up"], s["h"])
        return {"h": s["h"]}
    moe.moe_swiglu_backward(s["plan"], s["dh"], s["gate"], s["up"], s["dgate"], s["dup"], s["h"])
    return {"dgu": s["dgu"], "h": s["h"]}


def run(state):
    op = state["op"]
    if own:
        return (_own_linear if op == "linear" else _own_grouped if op == "grouped"
                else _own_swiglu)(state)
    return (_plain_linear if op == "linear" else _plain_grouped if op == "grouped"
            else _plain_swiglu)(state)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definitions in 64 bits."""
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()
         and k not in ("w", "gu")}
    out = {}
    if case["op"] == "swiglu":
        lim = case["limit"] if case["limit"] > 0 else math.inf
        g, u = torch.minimum(d["gate"], d["gate"].new_tensor(lim)), d["up"].clip(-lim, lim)
        e = torch.exp(-g)
        out["h"] = u * g / (1 + e)
        if case["back"]:
            slope = (1 + e + g * e) / (1 + e) ** 2  # of g / (1 + exp(-g))
            dg = torch.where(d["gate"] > lim, 0.0, d["dh"] * u * slope)
            du = torch.where((d["up"] > lim) | (d["up"] < -lim), 0.0, d["dh"] * g / (1 + e))
            out["dgu"] = torch.cat([dg, du], 1)
        return out
    if case["op"] == "linear":
        w = s["w"].double()
        value = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
        if not case["back"]:
            z = torch.addmm(d["b"], d["x"], w.t())
            out["y"] = value(z) + (d["r"] if case["residual"] else 0)
            if case["keep_z"]:
                out["z"] = z
            return out
        dz = d["dy"]
        if case["act"] != "none":
            z = d["z"].requires_grad_()
            dz, = torch.autograd.grad(value(z), z, d["dy"])
            out["dz"] = dz
        return {**out, "dx": torch.mm(dz, w), "dw": torch.mm(dz.t(), d["x"]), "db": dz.sum(0)}
    token = (s["pairs"] // case["per_token"]).long()
    x, at = d["x"].index_select(0, token), 0
    parts = {"y": [], "dx": [], "dw": [], "db": []}
    for e, m in enumerate(s["sizes"]):
        xe, we = x[at:at + m], s["w"][e].double()
        if not case["back"]:
            y = torch.mm(xe, we.t())
            parts["y"].append(y + d["b"][e] if case["bias"] else y)
        else:
            dy = d["dy"][at:at + m]
            parts["dx"].append(torch.mm(dy, we))
            parts["dw"].append(torch.mm(dy.t(), xe))
            parts["db"].append(dy.sum(0))
        at += m
    if not case["back"]:
        return {"y": torch.cat(parts["y"])}
    out = {"dx": torch.cat(parts["dx"]), "dw": torch.stack(parts["dw"])}
    return {**out, "db": torch.stack(parts["db"])} if case["bias"] else out
