"""What the operators around the expert products, and the products in 8 bits, are measured on.

Five operators:

* ``dispatch``: tokens' rows out to the experts in sorted order, r[pos[t][j]] = x[t], and its gradient
  dx[t] = base[t] + sum_j dr[pos[t][j]];
* ``combine``: the experts' rows back to the tokens, y[t] = base[t] + sum_j w[t][j] r[pos[t][j]], and its
  gradients dr[pos[t][j]] = w[t][j] dy[t] and dw[t][j] = <dy[t], r[pos[t][j]]>;
* ``quantize``: bf16 values to e4m3 codes with an fp32 scale for each block, of 1 x 128 (rows, which may go
  out to the experts on the way) or 128 x 128 (weights): a = max(largest magnitude, 2^-90), scale a / 448,
  code e4m3(x * 448 / a);
* ``linear_fp8``: y = act(x W^T + b) + residual with x and W in such codes and scales;
* ``grouped_fp8``: the experts' products in them, rows grouped by expert with ragged sizes.

A position pos[t][j] of -1 is a pair whose expert another GPU holds, or that was dropped. ``own`` chooses the
plain form in torch operations or the package's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK, MOST, LEAST = 128, 448.0, 2.0 ** -90


# ------------------------------------------------------------------ cases

def listed():
    return [
        # five decoded tokens sent out to their experts: latency
        dict(name="dispatch_decode", op="dispatch", back=False, tokens=5, per_token=8, hidden=4096,
             held=1.0, token="bf16", row="bf16", base=False),
        # the sum of a training batch's row gradients over each token's rows, added to the shared expert's
        dict(name="dispatch_back", op="dispatch", back=True, tokens=8192, per_token=8, hidden=4096,
             held=1.0, token="bf16", row="bf16", base=True),
        # a decode batch's weighted sum, beside the shared expert's output: latency
        dict(name="combine_decode", op="combine", back=False, tokens=64, per_token=8, hidden=4096,
             held=1.0, token="bf16", row="bf16", base=True),
        # a long prompt's, with fp32 outputs, on a GPU that holds about half of the experts
        dict(name="combine_long", op="combine", back=False, tokens=32768, per_token=8, hidden=4096,
             held=0.5, token="f32", row="bf16", base=False),
        # its backward pass in training, 48 experts at top 3, an odd batch
        dict(name="combine_back", op="combine", back=True, tokens=8191, per_token=3, hidden=7168,
             held=1.0, token="bf16", row="bf16", base=False),
        # the down product's operand of a prompt's routed rows, in 8 bits
        dict(name="quantize_rows", op="quantize", kind="rows", tokens=65536, per_token=1, cols=1280,
             held=1.0),
        # a prompt's tokens sent out to their experts in 8 bits
        dict(name="quantize_out", op="quantize", kind="out", tokens=8192, per_token=8, cols=4096, held=1.0),
        # one decoded token through a 4096 -> 1280 projection with everything in the epilogue: latency
        dict(name="linear_fp8_token", op="linear_fp8", rows=1, k=4096, n=1280, act="silu", residual=True,
             keep_z=False, out="bf16"),
        # a ragged prompt through odd widths (the last block of 128 holds 16) into fp32 logits
        dict(name="linear_fp8_odd", op="linear_fp8", rows=777, k=1296, n=2056, act="none", residual=False,
             keep_z=False, out="f32"),
        # a prompt through the dense layers' wide projection
        dict(name="linear_fp8_prefill", op="linear_fp8", rows=8192, k=4096, n=11264, act="none",
             residual=False, keep_z=False, out="bf16"),
        # a decode batch's gate product: 64 tokens on 8 of 288 experts each
        dict(name="grouped_fp8_decode", op="grouped_fp8", rows=512, groups=288, k=4096, n=1280, per_token=8,
             skew=1.0, bias=False, out="bf16"),
        # a prompt's gate product: 8192 tokens on 8 of 288 experts
        dict(name="grouped_fp8_prefill", op="grouped_fp8", rows=65536, groups=288, k=4096, n=1280,
             per_token=8, skew=0.5, bias=False, out="bf16"),
    ]


def _size(rng, low, high, step):
    """A multiple of `step` between low and high, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return int(min(high, max(low, round(v / step) * step)))


def draw(rng):
    while True:
        op = rng.choice(("dispatch", "combine", "quantize", "linear_fp8", "linear_fp8", "grouped_fp8"))
        k, n = _size(rng, 64, 11264, 16), _size(rng, 64, 11264, 8)
        kt = rng.choice((1, 2, 3, 4, 8))
        if op in ("dispatch", "combine"):
            back = rng.random() < 0.5
            c = dict(op=op, back=back, tokens=_size(rng, 1, 32768, 1), per_token=kt, hidden=n,
                     held=rng.choice((0.125, 0.5, 1.0)), token=rng.choice(("bf16", "f32")),
                     row=rng.choice(("bf16", "f32")), base=back == (op == "dispatch") and rng.random() < 0.5)
        elif op == "quantize":
            kind = rng.choice(("rows", "out", "weight"))
            c = dict(op=op, kind=kind, tokens=_size(rng, 1, 65536, 1), cols=k, held=1.0,
                     per_token=kt if kind == "out" else 1)
            if kind == "weight":  # tokens: the weights' rows, per_token: the number of weights
                c.update(tokens=n, per_token=_size(rng, 1, 288, 1))
            if kind == "out":
                c.update(held=rng.choice((0.125, 0.5, 1.0)))
        else:
            c = dict(op=op, rows=_size(rng, 1, 65536, 1), k=k, n=n, out=rng.choice(("bf16", "f32")))
            if op == "linear_fp8":
                act = rng.choice(ACTS)
                c.update(act=act, residual=rng.random() < 0.5,
                         keep_z=act != "none" and rng.random() < 0.5)
            else:
                c.update(groups=_size(rng, 2, 288, 1), per_token=kt, skew=rng.choice((0.0, 0.5, 1.0)),
                         bias=rng.random() < 0.5)
                if c["groups"] * k * n > 1_600_000_000:
                    continue
        w = work(c)
        if w["flops"] <= 7.6e11 and w["bytes"] <= 1.8e9:
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


def _held(case):
    """Pairs whose expert is held here."""
    return max(1, round(case["tokens"] * case["per_token"] * case["held"]))


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["op"] in ("dispatch", "combine"):
        t, h, r = case["tokens"], case["hidden"], _held(case)
        st, sr = (4 if case[x] == "f32" else 2 for x in ("token", "row"))
        pairs = t * case["per_token"]
        b = t * h * st * (2 if case["base"] else 1) + r * h * sr + 4 * pairs
        if case["op"] == "dispatch":
            return {"bytes": b, "flops": r * h * case["back"]}
        if not case["back"]:
            return {"bytes": b + 4 * pairs, "flops": 2 * r * h}
        return {"bytes": b + r * h * sr + 8 * pairs, "flops": 3 * r * h}
    if case["op"] == "quantize":
        t, c = case["tokens"], case["cols"]
        if case["kind"] == "weight":
            v = case["per_token"] * t * c
            return {"bytes": 3 * v + 4 * case["per_token"] * _blocks(t) * _blocks(c), "flops": 2 * v}
        r = _held(case) if case["kind"] == "out" else t
        return {"bytes": 2 * t * c + r * (c + 4 * _blocks(c)) + 4 * t * case["per_token"],
                "flops": 2 * t * c}
    p, k, n = case["rows"], case["k"], case["n"]
    f32 = 4 if case["out"] == "f32" else 2
    weight = n * k + 4 * _blocks(n) * _blocks(k)
    row = k + 4 * _blocks(k)
    if case["op"] == "linear_fp8":
        return {"bytes": p * row + weight + 4 * n + f32 * p * n
                + 2 * p * n * (case["residual"] + case["keep_z"]), "flops": 2 * p * n * k}
    active = sum(s > 0 for s in _group_sizes(case))
    return {"bytes": -(-p // case["per_token"]) * row + active * (weight + 4 * n * case["bias"])
            + f32 * p * n + 4 * p, "flops": 2 * p * n * k}


# ------------------------------------------------------------------ inputs

def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _codes(x, rows):
    """e4m3 codes and scales of [groups][n][k] in blocks of `rows` x 128, as a checkpoint holds them."""
    g, n, k = x.shape
    nb, kb = -(-n // rows), _blocks(k)
    v = torch.nn.functional.pad(x, (0, kb * BLOCK - k, 0, nb * rows - n)).float()
    v = v.view(g, nb, rows, kb, BLOCK)
    a = v.abs().amax((2, 4), keepdim=True).clamp(min=LEAST)
    q = (v * (MOST / a)).to(torch.float8_e4m3fn).view(g, nb * rows, kb * BLOCK)
    return q[:, :n, :k].contiguous(), (a / MOST).view(g, nb, kb)


def _positions(case, host):
    """Rows of the pairs held here, in the order of a stable sort by expert; -1 for the others."""
    pairs = case["tokens"] * case["per_token"]
    r = _held(case)
    expert = torch.randint(0, 288, (pairs,), generator=host)
    kept = torch.randperm(pairs, generator=host)[:r].sort().values
    order = kept[expert[kept].argsort(stable=True)]
    pos = torch.full((pairs,), -1, dtype=torch.int32)
    pos[order] = torch.arange(r, dtype=torch.int32)
    return pos.view(case["tokens"], case["per_token"])


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    host = torch.Generator().manual_seed(seed * 104729 + 11)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
        return t.mul_(scale) if scale != 1.0 else t

    s = dict(case)
    if case["op"] in ("dispatch", "combine"):
        t, kt, h, r = case["tokens"], case["per_token"], case["hidden"], _held(case)
        token, row = _dtype(case["token"]), _dtype(case["row"])
        s.update(pos=_positions(case, host).cuda(),
                 base=normal(t, h, dtype=token) if case["base"] else None)
        if case["op"] == "combine":
            w = torch.rand(t, kt, generator=g, device="cuda") + 0.05
            s.update(w=3.0 * w / w.sum(1, keepdim=True), r=normal(r, h, dtype=row))
            if case["back"]:
                s.update(dy=normal(t, h, scale=0.01, dtype=token))
        elif case["back"]:
            s.update(dr=normal(r, h, scale=0.01, dtype=row))
        else:
            s.update(x=normal(t, h, dtype=token))
        return s
    if case["op"] == "quantize":
        t, c = case["tokens"], case["cols"]
        if case["kind"] == "weight":
            s.update(x=normal(case["per_token"], t, c, scale=c ** -0.5))
        else:
            # rows whose sizes differ, as an activation's do
            size = torch.rand(t, 1, generator=g, device="cuda").mul_(6).sub_(3).exp2_()
            s.update(x=(normal(t, c) * size).to(torch.bfloat16),
                     pos=_positions(case, host).cuda() if case["kind"] == "out" else None)
        return s
    p, k, n = case["rows"], case["k"], case["n"]
    grouped = case["op"] == "grouped_fp8"
    e, kt = (case["groups"], case["per_token"]) if grouped else (1, 1)
    x8, xs = _codes(normal(1, -(-p // kt), k), 1)
    w8 = torch.empty((e, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    ws = torch.empty((e, _blocks(n), _blocks(k)), device="cuda")
    step = max(1, 100_000_000 // (n * k))
    for i in range(0, e, step):
        w8[i:i + step], ws[i:i + step] = _codes(normal(min(step, e - i), n, k, scale=k ** -0.5), BLOCK)
    s.update(x8=x8[0], xs=xs[0], w8=w8 if grouped else w8[0], ws=ws if grouped else ws[0])
    if not grouped:
        s.update(b=normal(n, scale=0.5, dtype=torch.float32), res=normal(p, n) if case["residual"] else None)
        return s
    sizes = torch.tensor(_group_sizes(case))[torch.randperm(e, generator=host)]
    # the pairs (token, slot) of each expert in ascending order, as a stable sort by expert leaves them
    pairs = torch.randperm(p, generator=host)
    pairs = torch.cat([t.sort().values for t in pairs.split(sizes.tolist())])
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)])
    s.update(sizes=sizes.tolist(), offsets=offsets.to(torch.int32).cuda(),
             pairs=pairs.to(torch.int32).cuda(),
             b=normal(e, n, scale=0.5, dtype=torch.float32) if case["bias"] else None)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    # the buffers that a program keeps for the outputs
    if case["op"] in ("dispatch", "combine"):
        t, h, r = case["tokens"], case["hidden"], _held(case)
        to_rows = case["back"] == (case["op"] == "combine")
        s.update(out=buf(r, h, dtype=_dtype(case["row"])) if to_rows
                 else buf(t, h, dtype=_dtype(case["token"])))
        if case["op"] == "combine" and case["back"]:
            s.update(dw=buf(t, case["per_token"], dtype=torch.float32))
    elif case["op"] == "quantize":
        t, c = case["tokens"], case["cols"]
        lead = {"rows": (t,), "out": (_held(case),), "weight": (case["per_token"], t)}[case["kind"]]
        blocks = (case["per_token"], _blocks(t)) if case["kind"] == "weight" else lead
        s.update(codes=buf(*lead, c, dtype=torch.float8_e4m3fn),
                 scales=buf(*blocks, _blocks(c), dtype=torch.float32))
    else:
        s.update(y=buf(case["rows"], case["n"], dtype=_dtype(case["out"])),
                 z=buf(case["rows"], case["n"]) if case.get("keep_z") else None)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_rows(s):
    """dispatch and combine."""
    held = s["pos"] >= 0
    pos = s["pos"].long().clamp(min=0)
    token, row = _dtype(s["token"]), _dtype(s["row"])
    if s["op"] == "dispatch" and not s["back"]:
        at = held.nonzero()
        r = torch.empty((_held(s), s["hidden"]), dtype=row, device=pos.device)
        r[pos[held]] = s["x"][at[:, 0]].to(row)
        return {"r": r}
    if s["op"] == "dispatch" or not s["back"]:
        v = s["dr" if s["back"] else "r"][pos].float() * held.unsqueeze(2)
        if s["op"] == "combine":
            v = v * s["w"].unsqueeze(2)
        y = v.sum(1)
        if s["base"] is not None:
            y = y + s["base"].float()
        return {"dx" if s["back"] else "y": y.to(token)}
    dy = s["dy"].float()
    dw = (s["r"][pos].float() * dy.unsqueeze(1)).sum(2) * held
    at = held.nonzero()
    dr = torch.empty((_held(s), s["hidden"]), dtype=row, device=pos.device)
    dr[pos[held]] = (dy[at[:, 0]] * s["w"][held].unsqueeze(1)).to(row)
    return {"dr": dr, "dw": dw}


def _plain_quantize(s):
    x = s["x"] if s["kind"] == "weight" else s["x"].unsqueeze(0)
    codes, scales = _codes(x, BLOCK if s["kind"] == "weight" else 1)
    if s["kind"] == "weight":
        return {"codes": codes, "scales": scales}
    codes, scales = codes[0], scales[0]
    if s["kind"] == "out":
        held = s["pos"] >= 0
        at, to = held.nonzero()[:, 0], s["pos"][held].long()
        c = torch.empty((_held(s), s["cols"]), dtype=torch.uint8, device=to.device)
        c[to] = codes.view(torch.uint8)[at]  # (torch indexes no 8-bit floats)
        sc = torch.empty((_held(s), scales.shape[1]), device=to.device)
        sc[to] = scales[at]
        codes, scales = c.view(torch.float8_e4m3fn), sc
    return {"codes": codes, "scales": scales}


def _values(codes, scales, rows):
    """The values that codes and their scales stand for, in fp32."""
    n, k = codes.shape
    sc = scales.repeat_interleave(rows, 0)[:n] if rows > 1 else scales
    return codes.float() * sc.repeat_interleave(BLOCK, 1)[:, :k]


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


def _plain_linear(s):
    z = _values(s["x8"], s["xs"], 1) @ _values(s["w8"], s["ws"], BLOCK).t() + s["b"]
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(_dtype(s["out"]))}
    if s["keep_z"]:
        out["z"] = z.to(torch.bfloat16)
    return out


def _plain_grouped(s):
    # one product per expert that has rows: ragged sizes leave torch no batched form of it
    x = _values(s["x8"], s["xs"], 1)[(s["pairs"] // s["per_token"]).long()]
    y = torch.empty((s["rows"], s["n"]), dtype=_dtype(s["out"]), device=x.device)
    at = 0
    for e, m in enumerate(s["sizes"]):
        if m:
            v = x[at:at + m] @ _values(s["w8"][e], s["ws"][e], BLOCK).t()
            y[at:at + m] = v + s["b"][e] if s["b"] is not None else v
        at += m
    return {"y": y}


# ------------------------------------------------------------------ the package's kernels

def _own_rows(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:  # a program makes the plan once
        s["plan"] = moe.make_dispatch_config(s["tokens"], _held(s), s["per_token"], s["hidden"],
                                             token_dtype=s["token"], row_dtype=s["row"])
    if s["op"] == "dispatch":
        if s["back"]:
            moe.moe_dispatch_backward(s["plan"], s["dr"], s["pos"], s["base"], s["out"])
            return {"dx": s["out"]}
        moe.moe_dispatch_forward(s["plan"], s["x"], s["pos"], s["out"])
        return {"r": s["out"]}
    if s["back"]:
        moe.moe_combine_backward(s["plan"], s["dy"], s["r"], s["pos"], s["w"], s["out"], s["dw"])
        return {"dr": s["out"], "dw": s["dw"]}
    moe.moe_combine_forward(s["plan"], s["r"], s["pos"], s["w"], s["base"], s["out"])
    return {"y": s["out"]}


def _own_quantize(s):
    import sparse_moe_layer_fp32_amd as moe
    if s["kind"] == "weight":
        moe.moe_quantize_weight(s["x"], s["codes"], s["scales"])
    else:
        if "plan" not in s:
            s["plan"] = moe.make_quantize_config(s["tokens"], s["cols"], rows=len(s["codes"]),
                                                 top_k=s["per_token"])
        moe.moe_quantize_rows(s["plan"], s["x"], s["pos"], s["codes"], s["scales"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_linear(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:  # and its workspace
        s["plan"] = moe.make_linear_config(s["rows"], s["k"], s["n"], activation=s["act"],
                                           y_dtype=s["out"])
        s["work"] = moe.alloc_linear_fp8_workspace(s["plan"])
    moe.moe_linear_forward_fp8(s["plan"], s["x8"], s["xs"], s["w8"], s["ws"], s["b"], s["res"], s["y"],
                               s["z"], s["work"])
    return {"y": s["y"], "z": s["z"]} if s["keep_z"] else {"y": s["y"]}


def _own_grouped(s):
    import sparse_moe_layer_fp32_amd as moe
    if "plan" not in s:
        s["plan"] = moe.make_grouped_config(s["rows"], s["groups"], s["k"], s["n"],
                                            x_rows=s["x8"].shape[0], row_div=s["per_token"],
                                            y_dtype=s["out"])
        s["work"] = moe.alloc_grouped_fp8_workspace(s["plan"])
    moe.moe_grouped_forward_fp8(s["plan"], s["x8"], s["xs"], s["pairs"], s["offsets"], s["w8"], s["ws"],
                                s["b"], s["y"], s["work"])
    return {"y": s["y"]}


def run(state):
    op = state["op"]
    if op in ("dispatch", "combine"):
        return (_own_rows if own else _plain_rows)(state)
    if op == "quantize":
        return (_own_quantize if own else _plain_quantize)(state)
    if op == "linear_fp8":
        return (_own_linear if own else _plain_linear)(state)
    return (_own_grouped if own else _plain_grouped)(state)


# ------------------------------------------------------------------ 64 bits

def _exact_block(x, rows):
    """codes and scales of one matrix, from the definition."""
    n, k = x.shape
    at = torch.arange(n, device=x.device).div(rows, rounding_mode="floor")
    blocks = [x[:, i:i + BLOCK].abs().amax(1) for i in range(0, k, BLOCK)]
    a = torch.stack(blocks, 1)
    if rows > 1:
        index = at.unsqueeze(1).expand_as(a)
        a = a.new_zeros(-(-n // rows), a.shape[1]).scatter_reduce(0, index, a, "amax")
    a = torch.maximum(a, a.new_tensor(LEAST))
    v = x * 448 / a[at][:, torch.arange(k, device=x.device) // BLOCK]
    # e4m3: three bits behind the first, steps of 2^-9 below 2^-6; torch.round takes ties to even
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    return torch.round(v / step) * step, a / 448


def exact(case, seed):
    """The definitions in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] in ("dispatch", "combine"):
        t, h, r = case["tokens"], case["hidden"], _held(case)
        pos = s["pos"].long()
        # the token and slot of each row
        pair = torch.zeros(r, dtype=torch.long, device=pos.device)
        flat = pos.flatten()
        which = (flat >= 0).nonzero().flatten()
        pair[flat[which]] = which
        token = pair // case["per_token"]
        if case["op"] == "dispatch" and not case["back"]:
            return {"r": s["x"].double().index_select(0, token)}
        if case["op"] == "combine" and case["back"]:
            dy = s["dy"].double().index_select(0, token)
            w = s["w"].double().flatten()
            dw = torch.zeros_like(w)
            dw[pair] = (dy * s["r"].double()).sum(1)
            return {"dr": dy * w[pair].unsqueeze(1), "dw": dw.view(t, case["per_token"])}
        y = s["base"].double() if case["base"] else torch.zeros((t, h), dtype=torch.double, device=pos.device)
        rows = s["dr"] if case["back"] else s["r"]
        for j in range(case["per_token"]):
            at = (pos[:, j] >= 0).nonzero().flatten()
            v = rows[pos[at, j]].double()
            y[at] += v if case["back"] else v * s["w"][at, j].double().unsqueeze(1)
        return {"dx" if case["back"] else "y": y}
    if case["op"] == "quantize":
        if case["kind"] == "weight":
            pairs = [_exact_block(w.double(), BLOCK) for w in s["x"]]
            return {"codes": torch.stack([c for c, _ in pairs]), "scales": torch.stack([a for _, a in pairs])}
        codes, scales = _exact_block(s["x"].double(), 1)
        if case["kind"] == "out":
            flat = s["pos"].flatten().long()
            which = (flat >= 0).nonzero().flatten()
            token = torch.empty_like(which)
            token[flat[which]] = which // case["per_token"]
            codes, scales = codes.index_select(0, token), scales.index_select(0, token)
        return {"codes": codes, "scales": scales}
    k, n = case["k"], case["n"]
    kb = torch.arange(k, device="cuda") // BLOCK
    fb = torch.arange(n, device="cuda") // BLOCK
    x = s["x8"].double() * s["xs"].double()[:, kb]
    weight = lambda w, sc: w.double().mul_(sc.double()[fb][:, kb])  # noqa: E731
    if case["op"] == "linear_fp8":
        value = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
        z = torch.addmm(s["b"].double(), x, weight(s["w8"], s["ws"]).t())
        y = value(z) + (s["res"].double() if case["residual"] else 0)
        return {"y": y, "z": z} if case["keep_z"] else {"y": y}
    x, at, parts = x.index_select(0, (s["pairs"] // case["per_token"]).long()), 0, []
    for e, m in enumerate(s["sizes"]):
        y = torch.mm(x[at:at + m], weight(s["w8"][e], s["ws"][e]).t())
        parts.append(y + s["b"][e].double() if case["bias"] else y)
        at += m
    return {"y": torch.cat(parts)}
