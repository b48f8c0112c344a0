"""The operators beside the MoE layer as they are measured: their cases, their
inputs, their plain forms in elementary torch operations, and their definitions
in 64 bits.

  join     norms before and after a block, with its gate and residual scale
  grouped  products grouped by expert over ragged groups of rows
  adapter  a shared projection with one low-rank adapter per token

`run` computes the plain form where `own` is false and calls the library where
it is true. Inputs depend on the case and the seed alone.
"""
import math
import random

import torch

own = False

EPS = 1e-6
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token of the 4096-wide layer: the cost of a call
        {"name": "join 1x4096", "op": "join", "way": "forward", "m": 1, "dim": 4096, "type": "bf16",
         "res": "bf16", "gate": "shared", "post": True},
        # a long prompt, residual stream kept in 32 bits
        {"name": "join 8192x4096", "op": "join", "way": "forward", "m": 8192, "dim": 4096, "type": "bf16",
         "res": "f32", "gate": "shared", "post": True},
        # its training step: gradients of the shared gate and of both norm weights are sums over the rows
        {"name": "join back 4096x4096", "op": "join", "way": "backward", "m": 4096, "dim": 4096, "type": "bf16",
         "res": "bf16", "gate": "shared", "post": True},
        # a width that no vector load divides, a gate per token
        {"name": "join back 777x1001", "op": "join", "way": "backward", "m": 777, "dim": 1001, "type": "fp16",
         "res": "fp16", "gate": "rows", "post": True},
        # 8 decoded tokens with 6 picks each: 48 rows over 384 experts, most groups empty
        {"name": "grouped 48 of 384", "op": "grouped", "way": "forward", "groups": 384, "rows": 48, "n": 2048,
         "k": 4096, "skew": 0.3, "type": "bf16", "out": "bf16"},
        # a 2048-token prompt with 6 picks each over all experts: about 32 rows a group, ragged
        {"name": "grouped 12288 of 384", "op": "grouped", "way": "forward", "groups": 384, "rows": 12288, "n": 2048,
         "k": 4096, "skew": 0.5, "type": "bf16", "out": "bf16"},
        # a training batch on the experts of one rank, through the down projection's input gradient
        {"name": "grouped dx 16384 of 32", "op": "grouped", "way": "dx", "groups": 32, "rows": 16384, "n": 4096,
         "k": 2048, "skew": 0.4, "type": "fp16", "out": "fp16"},
        # and its weight gradient, kept in 32 bits for the optimizer
        {"name": "grouped dw 16384 of 32", "op": "grouped", "way": "dw", "groups": 32, "rows": 16384, "n": 4096,
         "k": 2048, "skew": 0.4, "type": "bf16", "out": "f32"},
        # a small layer with odd widths: rows that start at odd addresses
        {"name": "grouped dw 1000 odd", "op": "grouped", "way": "dw", "groups": 13, "rows": 1000, "n": 257,
         "k": 515, "skew": 0.8, "type": "bf16", "out": "bf16"},
        # one decoded token with its request's adapter on the shared expert's up projection
        {"name": "adapter 1 token", "op": "adapter", "m": 1, "n": 2048, "k": 4096, "rank": 16, "adapters": 8,
         "order": "mixed", "type": "bf16", "out": "bf16"},
        # a decode batch: every token another request, 24 adapters among them
        {"name": "adapter 48 tokens", "op": "adapter", "m": 48, "n": 2048, "k": 4096, "rank": 32, "adapters": 24,
         "order": "mixed", "type": "fp16", "out": "fp16"},
        # prompts of 8 requests one after another, through the down projection
        {"name": "adapter 4096 tokens", "op": "adapter", "m": 4096, "n": 4096, "k": 2048, "rank": 64, "adapters": 8,
         "order": "segments", "type": "bf16", "out": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A width: mostly multiples of 64 as models have them, sometimes any number."""
    v = _spread(rng, lo, hi)
    v = max(64, 64 * round(v / 64)) if rng.random() < 0.75 else v
    return v - 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["join", "grouped", "adapter"])
    t = rng.choice(["bf16", "fp16"])
    if op == "join":
        return {"op": op, "way": rng.choice(["forward", "backward"]), "m": _spread(rng, 1, 8192),
                "dim": _width(rng, 100, 4096), "type": t, "res": rng.choice([t, "f32"]),
                "gate": rng.choice(["none", "shared", "rows"]), "post": rng.random() < 0.75}
    if op == "grouped":
        groups = _spread(rng, 1, 128)
        rows = _spread(rng, 1, 12000)
        return {"op": op, "way": rng.choice(["forward", "dx", "dw"]), "groups": groups, "rows": rows - (rows == 3072),
                "n": _width(rng, 64, 4096), "k": _width(rng, 64, 2048), "skew": round(rng.uniform(0.0, 1.0), 2),
                "type": t, "out": rng.choice([t, t, "f32"])}
    m = _spread(rng, 1, 4096)
    return {"op": op, "m": m - (m == 3072), "n": _width(rng, 64, 4096), "k": _width(rng, 64, 4096),
            "rank": _spread(rng, 1, 64), "adapters": _spread(rng, 1, 32), "order": rng.choice(["mixed", "segments"]),
            "type": t, "out": rng.choice([t, t, "f32"])}


def _sizes(rows, groups, skew):
    """Rows of each group, largest first: group i's share falls as (i + 1)^-skew."""
    w = [(i + 1.0) ** -skew for i in range(groups)]
    sizes = [int(rows * v / sum(w)) for v in w]
    for i in range(rows - sum(sizes)):
        sizes[i % groups] += 1
    return sizes


def _row_sizes(case, seed):
    """The groups' sizes in the seed's order."""
    sizes = _sizes(case["rows"], case["groups"], case["skew"])
    random.Random(seed).shuffle(sizes)
    return sizes


def _adapter_sizes(case):
    """Rows of each adapter, and of none (an eighth of them)."""
    bare = case["m"] // 8
    return _sizes(case["m"] - bare, case["adapters"], 0.3), bare


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _normal(gen, shape, dtype, sigma=1.0, mean=0.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(sigma).add_(mean)


def _inputs(case, seed):
    gen, t = _gen(seed), _TYPES[case["type"]]
    if case["op"] == "join":
        m, dim, res = case["m"], case["dim"], _TYPES[case["res"]]
        s = {"x": _normal(gen, (m, dim), res, 2.0), "block": _normal(gen, (m, dim), t),
             "w_post": _normal(gen, (dim,), t, 0.2, 1.0) if case["post"] else None,
             "w_pre": _normal(gen, (dim,), t, 0.2, 1.0), "gate": None, "scale": 0.7}
        if case["gate"] != "none":
            s["gate"] = _normal(gen, (m, dim) if case["gate"] == "rows" else (dim,), t, 0.3, 0.5)
        if case["way"] == "backward":
            # x holds what the forward pass wrote: the stream after the block
            s["dy"] = _normal(gen, (m, dim), t)
            s["dx_out"] = _normal(gen, (m, dim), res)
        return s
    if case["op"] == "grouped":
        n, k, rows, sizes = case["n"], case["k"], case["rows"], _row_sizes(case, seed)
        bounds = [0]
        for v in sizes:
            bounds.append(bounds[-1] + v)
        s = {"offsets": torch.tensor(bounds, dtype=torch.int32, device="cuda"), "most": max(sizes)}
        if case["way"] != "dw":
            s["w"] = _normal(gen, (case["groups"], n, k), t, 0.02)
        if case["way"] != "forward":
            s["dy"] = _normal(gen, (rows, n), t)
        if case["way"] != "dx":
            s["x"] = _normal(gen, (rows, k), t)
        return s
    m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
    sizes, bare = _adapter_sizes(case)
    order = list(range(case["adapters"])) + [-1]
    sizes = sizes + [bare]
    rnd = random.Random(seed)
    rnd.shuffle(order)
    index = [a for a in order for _ in range(sizes[a])]
    if case["order"] == "mixed":
        rnd.shuffle(index)
    return {"x": _normal(gen, (m, k), t), "w": _normal(gen, (n, k), t, 0.02),
            "a": _normal(gen, (case["adapters"], r, k), t, 0.02), "b": _normal(gen, (case["adapters"], n, r), t, 0.05),
            "factor": torch.rand(case["adapters"], generator=gen, device="cuda") * 1.5 + 0.5,
            "index": torch.tensor(index, dtype=torch.int32, device="cuda")}


def _handles(case, s):
    """What a program that uses the library keeps: the description of the call, its output buffers and workspace."""
    import routing_quant_expert_amd as R

    def like(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    t = _TYPES[case["type"]]
    if case["op"] == "join":
        m, dim = case["m"], case["dim"]
        h = {"plan": R.Join(dim, t, residual=_TYPES[case["res"]], gate_rows=case["gate"] == "rows", scale=s["scale"],
                            eps=EPS)}
        if case["way"] == "forward":
            return {**h, "x_out": torch.empty_like(s["x"]), "y": like((m, dim), t)}
        return {**h, "dx": torch.empty_like(s["x"]), "dblock": like((m, dim), t),
                "dw_post": like((dim,), torch.float32) if case["post"] else None, "dw_pre": like((dim,), torch.float32),
                "dgate": None if case["gate"] == "none" else like((m, dim), t) if case["gate"] == "rows"
                else like((dim,), torch.float32),
                "ws": like((R.join_workspace_bytes(h["plan"], m),), torch.uint8)}
    out = _TYPES[case["out"]]
    if case["op"] == "grouped":
        shape = {"forward": (case["rows"], case["n"]), "dx": (case["rows"], case["k"]),
                 "dw": (case["groups"], case["n"], case["k"])}[case["way"]]
        return {"plan": R.Grouped(case["groups"], case["n"], case["k"], t, out=out), "out": like(shape, out)}
    plan = R.Adapters(s["a"], s["b"], s["factor"], out=out)
    return {"plan": plan, "out": like((case["m"], case["n"]), out),
            "ws": like((R.adapter_workspace_bytes(plan, case["m"]),), torch.uint8)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s.update(_handles(case, s))
    return s


def _run_own(s):
    import routing_quant_expert_amd as R

    case = s["case"]
    if case["op"] == "join":
        if case["way"] == "forward":
            R.join_forward(s["plan"], s["x"], s["block"], s["w_post"], s["gate"], s["w_pre"], s["x_out"], s["y"])
            return {"x_out": s["x_out"], "y": s["y"]}
        R.join_backward(s["plan"], s["dy"], s["dx_out"], s["x"], s["block"], s["w_post"], s["gate"], s["w_pre"],
                        s["dx"], s["dblock"], s["dw_post"], s["dgate"], s["dw_pre"], s["ws"])
        return {k: s[k] for k in ("dx", "dblock", "dw_post", "dgate", "dw_pre") if s[k] is not None}
    if case["op"] == "grouped":
        if case["way"] == "forward":
            R.grouped_forward(s["plan"], s["x"], s["w"], s["offsets"], s["out"])
        elif case["way"] == "dx":
            R.grouped_backward_x(s["plan"], s["dy"], s["w"], s["offsets"], s["out"])
        else:
            R.grouped_backward_w(s["plan"], s["dy"], s["x"], s["offsets"], s["out"])
        return s["out"]
    R.adapter_project(s["plan"], s["x"], s["w"], s["index"], s["out"], s["ws"])
    return s["out"]


def _plain_join(s, case):
    t, res = _TYPES[case["type"]], _TYPES[case["res"]]
    x, block, w_pre = s["x"].float(), s["block"].float(), s["w_pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    rb = torch.rsqrt(block.square().mean(-1, keepdim=True) + EPS) if case["post"] else None
    nb = block * rb if case["post"] else block
    z = nb * s["w_post"].float() if case["post"] else nb
    if case["way"] == "forward":
        x = x + s["scale"] * (gate * z)
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w_pre
        return {"x_out": x.to(res), "y": y.to(t)}
    dy = s["dy"].float()
    rx = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * rx
    dn = dy * w_pre
    dx = s["dx_out"].float() + rx * (dn - n * (dn * n).mean(-1, keepdim=True))
    dz = s["scale"] * (gate * dx)
    out = {"dx": dx.to(res), "dw_pre": (dy * n).sum(0)}
    if case["post"]:
        dnb = dz * s["w_post"].float()
        out["dblock"] = (rb * (dnb - nb * (dnb * nb).mean(-1, keepdim=True))).to(t)
        out["dw_post"] = (dz * nb).sum(0)
    else:
        out["dblock"] = dz.to(t)
    if case["gate"] == "rows":
        out["dgate"] = (s["scale"] * dx * z).to(t)
    elif case["gate"] == "shared":
        out["dgate"] = (s["scale"] * dx * z).sum(0)
    return out


def _plain_grouped(s, case):
    """Few rows: each row with its own group's weight. Otherwise every group padded to the largest."""
    off, rows, groups = s["offsets"], case["rows"], case["groups"]
    out = _TYPES[case["out"]]
    way = case["way"]
    gid = torch.searchsorted(off[1:], torch.arange(rows, dtype=torch.int32, device="cuda"), right=True)
    if way != "dw" and rows < groups:
        w = s["w"][gid].float()
        if way == "forward":
            return torch.bmm(w, s["x"].float()[:, :, None])[:, :, 0].to(out)
        return torch.bmm(s["dy"].float()[:, None, :], w)[:, 0].to(out)
    place = gid * s["most"] + torch.arange(rows, device="cuda") - off[gid]

    def padded(v):
        p = torch.zeros((groups * s["most"], v.shape[1]), dtype=torch.float32, device="cuda")
        p[place] = v.float()
        return p.view(groups, s["most"], v.shape[1])

    if way == "forward":
        return torch.bmm(padded(s["x"]), s["w"].float().transpose(1, 2)).view(-1, case["n"])[place].to(out)
    if way == "dx":
        return torch.bmm(padded(s["dy"]), s["w"].float()).view(-1, case["k"])[place].to(out)
    return torch.bmm(padded(s["dy"]).transpose(1, 2), padded(s["x"])).to(out)


def _plain_adapter(s, case):
    """All adapters' low-rank products for every token, those of other adapters zeroed."""
    x, na, r = s["x"].float(), case["adapters"], case["rank"]
    mine = (s["index"][:, None] == torch.arange(na, dtype=torch.int32, device="cuda")) * s["factor"]
    u = (x @ s["a"].float().view(na * r, case["k"]).t()).view(-1, na, r) * mine[:, :, None]
    b = s["b"].float().transpose(1, 2).reshape(na * r, case["n"])
    return (x @ s["w"].float().t() + u.view(-1, na * r) @ b).to(_TYPES[case["out"]])


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    return {"join": _plain_join, "grouped": _plain_grouped, "adapter": _plain_adapter}[case["op"]](state, case)


def work(case):
    e = 2   # bytes of bf16 and fp16
    if case["op"] == "join":
        m, dim = case["m"], case["dim"]
        r = 4 if case["res"] == "f32" else 2
        per = r + e                                        # x and the block's output, read
        per += e if case["gate"] == "rows" else 0          # a gate per token, read
        if case["way"] == "forward":
            per += r + e                                   # the stream and the norm, written
            return {"bytes": m * dim * per + 3 * dim * e, "flops": 12 * m * dim}
        per += e + r + r + e                               # dy and dx_out read, dx and dblock written
        per += e if case["gate"] == "rows" else 0          # the gate's gradient
        return {"bytes": m * dim * per + dim * (3 * e + 3 * 4), "flops": 30 * m * dim}
    o = 4 if case["out"] == "f32" else 2
    n, k = case["n"], case["k"]
    if case["op"] == "grouped":
        rows, used = case["rows"], sum(v > 0 for v in _sizes(case["rows"], case["groups"], case["skew"]))
        moved = {"forward": rows * k * e + used * n * k * e + rows * n * o,
                 "dx": rows * n * e + used * n * k * e + rows * k * o,
                 "dw": rows * (n + k) * e + case["groups"] * n * k * o}[case["way"]]
        return {"bytes": moved + 4 * (case["groups"] + 1), "flops": 2.0 * rows * n * k}
    sizes, bare = _adapter_sizes(case)
    m, r, used = case["m"], case["rank"], sum(v > 0 for v in sizes)
    return {"bytes": m * k * e + n * k * e + used * (r * (n + k) * e + 4) + 4 * m + m * n * o,
            "flops": 2.0 * m * n * k + 2.0 * (m - bare) * r * (n + k)}


def exact(case, seed):
    """The operators' definitions, row by row and group by group, in 64 bits."""
    s = _inputs(case, seed)
    f = {key: v.double() if torch.is_tensor(v) and v.is_floating_point() and v.dim() < 3 else v
         for key, v in s.items()}
    if case["op"] == "join":
        def norm(v):
            return (v.pow(2).sum(1) / v.shape[1] + EPS).pow(-0.5)[:, None]

        gain = torch.ones_like(f["block"]) if f["gate"] is None else f["gate"].expand_as(f["block"])
        gain = gain * s["scale"]
        post = f["w_post"] if case["post"] else torch.ones_like(f["w_pre"])
        rb = norm(f["block"]) if case["post"] else torch.ones_like(f["block"][:, :1])
        if case["way"] == "forward":
            stream = f["x"] + gain * post * f["block"] * rb
            return {"x_out": stream, "y": stream * norm(stream) * f["w_pre"]}
        rx = norm(f["x"])
        # d(v_i r)/dv_j = r (delta_ij - v_i v_j r^2 / dim)
        g = f["dy"] * f["w_pre"]
        dx = f["dx_out"] + rx * g - f["x"] * rx.pow(3) * (g * f["x"]).sum(1, keepdim=True) / case["dim"]
        out = {"dx": dx, "dw_pre": (f["dy"] * f["x"] * rx).sum(0)}
        h = dx * gain * post
        if case["post"]:
            b = f["block"]
            out["dblock"] = rb * h - b * rb.pow(3) * (h * b).sum(1, keepdim=True) / case["dim"]
            out["dw_post"] = (dx * gain * b * rb).sum(0)
        else:
            out["dblock"] = h
        if case["gate"] != "none":
            dg = s["scale"] * dx * post * f["block"] * rb
            out["dgate"] = dg if case["gate"] == "rows" else dg.sum(0)
        return out
    if case["op"] == "grouped":
        ends = s["offsets"].tolist()
        shape = {"forward": (case["rows"], case["n"]), "dx": (case["rows"], case["k"]),
                 "dw": (case["groups"], case["n"], case["k"])}[case["way"]]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for g in range(case["groups"]):
            a, b = ends[g], ends[g + 1]
            if a == b:
                continue
            if case["way"] == "forward":
                out[a:b] = f["x"][a:b] @ s["w"][g].double().t()
            elif case["way"] == "dx":
                out[a:b] = f["dy"][a:b] @ s["w"][g].double()
            else:
                out[g] = f["dy"][a:b].t() @ f["x"][a:b]
        return out
    out = f["x"] @ f["w"].t()
    for a in range(case["adapters"]):
        rows = (s["index"] == a).nonzero()[:, 0]
        if rows.numel():
            low = f["x"][rows] @ s["a"][a].double().t()
            out[rows] += f["factor"][a] * (low @ s["b"][a].double().t())
    return out
