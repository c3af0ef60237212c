"""What is measured of the operators that serve a mixture of experts, and plain linear layers, from 4-bit weights.

Four of them, as a server runs them in a feed-forward step:

  linear   Y = X W^T for W in 4 bits with a scale (and a zero) per group of a row's elements: one token, a batch of them,
           a long prompt
  route    the experts of each token from its router's logits: the top k of them, their weights, and the tokens' places
           in an order by expert
  experts  the products of the tokens of each expert with that expert's 4-bit matrix, ragged: `up` takes each token's row
           of X and ends in silu(gate) * up of row pairs, `down` takes the rows in the experts' order
  combine  each token's weighted sum of its experts' rows, added to the residual stream

A matrix is codes [experts][rows][cols / 2] (element k in byte k / 2, the low four bits first), scales and zeros
[experts][rows][groups]: element k of a row is scales[k / group] * (code - zeros[k / group]), zeros 8 where there are none.
Slot i of the order holds pick order[i] = token * top_k + j; those of expert e are offsets[e] .. offsets[e + 1].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through a wide projection, the 12,288 x 1,536 matrix that the framework's GEMVs are quoted on: a latency
        dict(name="linear 1 x 1536 to 12288", op="linear", tokens=1, cols=1536, rows=12288, group=128, zeros=False,
             dtype="f16", out="f32"),
        # the same transposed, in small groups: few rows, so K is cut over the GPU
        dict(name="linear 1 x 12288 to 1536", op="linear", tokens=1, cols=12288, rows=1536, group=32, zeros=True,
             dtype="bf16", out="f32"),
        # a batch of answers
        dict(name="linear 13 x 4096 to 10240", op="linear", tokens=13, cols=4096, rows=10240, group=64, zeros=True,
             dtype="f16", out="f16"),
        # a short prompt through a small model's attention projection, columns that end inside a group
        dict(name="linear 222 x 776 to 2304", op="linear", tokens=222, cols=776, rows=2304, group=128, zeros=False,
             dtype="f16", out="f32"),
        # a long prompt: the matrix products bound it
        dict(name="linear 4096 x 4096 to 8192", op="linear", tokens=4096, cols=4096, rows=8192, group=128, zeros=True,
             dtype="bf16", out="bf16"),
        # one token's experts: a latency
        dict(name="route 1 x 8", op="route", tokens=1, experts=8, top_k=2, score="softmax", renorm=True, dtype="f32"),
        # a batch of prompts over many experts
        dict(name="route 8191 x 128", op="route", tokens=8191, experts=128, top_k=8, score="sigmoid", renorm=True,
             dtype="bf16"),
        # one token, two of eight experts
        dict(name="experts up 1 of 8", op="up", tokens=1, experts=8, top_k=2, cols=2048, rows=8192, group=128, zeros=False,
             dtype="bf16", out="bf16"),
        # a batch's step over many small experts: every expert has a few tokens
        dict(name="experts down 64 of 64", op="down", tokens=64, experts=64, top_k=8, cols=1408, rows=2048, group=64,
             zeros=True, dtype="f16", out="f32"),
        # a long prompt over a few large experts
        dict(name="experts up 4096 of 8", op="up", tokens=4096, experts=8, top_k=2, cols=2048, rows=8192, group=128,
             zeros=False, dtype="bf16", out="bf16"),
        # a batch's step
        dict(name="combine 64 x 2048", op="combine", tokens=64, top_k=8, cols=2048, dtype="f32", out="f32"),
        # a batch of prompts
        dict(name="combine 8191 x 2048", op="combine", tokens=8191, top_k=8, cols=2048, dtype="f32", out="bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "up", "down", "up", "down", "route", "combine"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "route":
        experts = _log(rng, 4, 256)
        return dict(op="route", tokens=_log(rng, 1, 8191), experts=experts, top_k=rng.randint(1, min(8, experts)),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5, dtype=rng.choice(["f16", "bf16", "f32"]))
    if op == "combine":
        return dict(op="combine", tokens=_log(rng, 1, 8191), top_k=rng.randint(1, 8), cols=8 * _log(rng, 64, 256),
                    dtype=rng.choice(["f32", dtype]), out=rng.choice(["f32", dtype]))
    case = dict(op=op, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, dtype=dtype, out=rng.choice(["f32", dtype]))
    if op == "linear":
        cols = 8 * _log(rng, 64, 1536)
        return dict(case, tokens=_log(rng, 1, 2048), cols=cols, rows=2 * _log(rng, 256, 6144 if cols <= 4096 else 2048))
    experts = _log(rng, 4, 64)
    return dict(case, tokens=_log(rng, 1, 2048), experts=experts, top_k=rng.randint(1, min(8, experts) // 2),
                cols=8 * _log(rng, 64, 256), rows=2 * _log(rng, 128, 1024))


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    t = case["tokens"]
    if case["op"] == "route":
        n, k = t * case["experts"], t * case["top_k"]
        return {"bytes": n * size[case["dtype"]] + 16 * k + 4 * case["experts"], "flops": 4 * n}
    if case["op"] == "combine":
        n = t * case["cols"]
        return {"bytes": n * (case["top_k"] * size[case["dtype"]] + 2 * size[case["out"]]) + 8 * t * case["top_k"],
                "flops": 2 * n * case["top_k"]}
    k, rows, groups = case["cols"], case["rows"], -(-case["cols"] // case["group"])
    matrix = rows * (k / 2 + groups * (3 if case["zeros"] else 2))
    if case["op"] == "linear":
        return {"bytes": int(matrix + 2 * t * k + size[case["out"]] * t * rows), "flops": 2 * t * k * rows}
    slots = t * case["top_k"]
    used = case["experts"] * (1 - (1 - case["top_k"] / case["experts"]) ** t)  # experts that some token goes to
    x, y = (t, rows // 2) if case["op"] == "up" else (slots, rows)
    return {"bytes": int(used * matrix + 2 * x * k + size[case["out"]] * slots * y + 4 * slots), "flops": 2 * slots * k * rows}


# ------------------------------------------------------------------ what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def logits(dtype):  # some experts are liked more than others
        return (normal(case["tokens"], case["experts"]) + normal(case["experts"], scale=0.5)).to(dtype)

    dtype, t = FLOATS[case["dtype"]], case["tokens"]
    state = dict(op=case["op"], tokens=t)
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        empty = lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
        return dict(state, logits=logits(dtype), experts=e, top_k=k, score=case["score"], renorm=case["renorm"], scale=1.0,
                    ids=empty(t, k), weights=empty(t, k, dtype=torch.float32), offsets=empty(e + 1), order=empty(t * k),
                    slots=empty(t, k))
    if case["op"] == "combine":
        k, n = case["top_k"], case["cols"]
        weights = torch.rand(t, k, generator=g, device=DEV)
        # in the order of experts a token's rows lie apart
        return dict(state, y=normal(t * k, n, dtype=dtype), slots=torch.randperm(t * k, generator=g, device=DEV).int().view(t, k),
                    weights=weights / weights.sum(1, keepdim=True), residual=normal(t, n, dtype=FLOATS[case["out"]]),
                    out=torch.empty(t, n, dtype=FLOATS[case["out"]], device=DEV), top_k=k)
    e, rows, cols, group = case.get("experts", 1), case["rows"], case["cols"], case["group"]
    groups, wide = -(-cols // group), 32 * -(-cols // 32)  # rows of codes start at 16 bytes
    code = [(normal(e, rows, wide // 2, scale=3.0) + 8).round_().clamp_(0, 15).to(torch.uint8) for _ in range(2)]
    state |= dict(codes=code[0] | code[1] << 4, cols=cols, rows=rows, group=group,
                  scales=(0.33 / math.sqrt(cols) * (0.8 + 0.4 * torch.rand(e, rows, groups, generator=g, device=DEV))).to(dtype),
                  zeros=torch.randint(6, 11, (e, rows, groups), generator=g, device=DEV, dtype=torch.uint8) if case["zeros"] else None)
    if case["op"] == "linear":
        return dict(state, x=normal(t, cols, dtype=dtype), y=torch.empty(t, rows, dtype=FLOATS[case["out"]], device=DEV))
    k, n = case["top_k"], t * case["top_k"]
    ids = logits(torch.float32).topk(k, 1).indices.reshape(-1)
    order = ids.sort(stable=True).indices.int()
    counts = torch.bincount(ids, minlength=e)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    up = case["op"] == "up"
    return dict(state, x=normal(t if up else n, cols, dtype=dtype), order=order, offsets=offsets, top_k=k, n=n,
                experts=e, most=int(counts.max()), y=torch.empty(n, rows // 2 if up else rows, dtype=FLOATS[case["out"]], device=DEV))


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "route": _plain_route, "up": _plain_experts, "down": _plain_experts,
            "combine": _plain_combine}[state["op"]](state)


def _own(s):
    import dense_packed_bit_gb300 as mm
    op, t = s["op"], s["tokens"]
    if op == "route":
        ws = s.get("workspace")
        if ws is None:
            n = mm.mm_experts_route_workspace(t, s["experts"], s["top_k"])
            ws = s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
        mm.mm_experts_route(s["logits"], t, s["experts"], s["logits"].stride(0), s["top_k"],
                            mm.MM_ROUTE_SIGMOID if s["score"] == "sigmoid" else mm.MM_ROUTE_SOFTMAX, s["renorm"], s["scale"],
                            s["ids"], s["weights"], s["offsets"], s["order"], s["slots"], ws, ws.numel())
        return {x: s[x] for x in ("ids", "weights", "offsets", "order", "slots")}
    if op == "combine":
        mm.mm_experts_combine(s["y"], s["y"].stride(0), s["y"].shape[0], s["slots"], s["weights"], t, s["top_k"], s["y"].shape[1],
                              s["residual"], s["residual"].stride(0), s["out"], s["out"].stride(0))
        return s["out"]
    w = s.get("w")
    if w is None:
        w = s["w"] = mm.mm_packed4(s["codes"], s["scales"], s["zeros"], s["cols"], s["group"], weights_static=True)
    if op == "linear":
        mm.mm_gemm_packed4(w, s["x"], s["x"].stride(0), t, mm.MM_ACT_NONE, s["y"], s["y"].stride(0))
    elif op == "up":
        mm.mm_experts_gemm_packed4(w, s["x"], s["x"].stride(0), t, s["order"], s["top_k"], s["offsets"], s["n"], mm.MM_ACT_SWIGLU,
                                   s["y"], s["y"].stride(0))
    else:
        mm.mm_experts_gemm_packed4(w, s["x"], s["x"].stride(0), s["n"], None, 1, s["offsets"], s["n"], mm.MM_ACT_NONE, s["y"],
                                   s["y"].stride(0))
    return s["y"]


def _matrix(codes, scales, zeros, cols, group):
    """[...][rows][cols] in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :cols].float()
    each = lambda a: a.float().repeat_interleave(group, -1)[..., :cols]  # noqa: E731
    return (code - (8.0 if zeros is None else each(zeros))).mul_(each(scales))


def _plain_linear(s):
    w = _matrix(s["codes"][0], s["scales"][0], None if s["zeros"] is None else s["zeros"][0], s["cols"], s["group"])
    s["y"].copy_(s["x"].float() @ w.T)
    return s["y"]


def _plain_route(s):
    x, k = s["logits"].float(), s["top_k"]
    x = x.masked_fill(torch.isnan(x), -math.inf)
    ids = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    weights = score.gather(1, ids)
    if s["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    order = flat.sort(stable=True).indices
    counts = torch.zeros(s["experts"], dtype=torch.int64, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))
    s["ids"].copy_(ids)
    s["weights"].copy_(weights * s["scale"])
    s["offsets"][0] = 0
    s["offsets"][1:] = counts.cumsum(0)
    s["order"].copy_(order)
    s["slots"].view(-1)[order] = torch.arange(flat.shape[0], dtype=torch.int32, device=x.device)
    return {x: s[x] for x in ("ids", "weights", "offsets", "order", "slots")}


def _plain_experts(s):
    n, e, offsets = s["n"], s["experts"], s["offsets"].long()
    i = torch.arange(n, device=DEV)
    of = torch.searchsorted(offsets, i, right=True) - 1  # the expert of each slot
    x = (s["x"][s["order"].long() // s["top_k"]] if s["op"] == "up" else s["x"]).float()
    if n <= e:  # each slot with its own expert's matrix
        w = _matrix(s["codes"][of], s["scales"][of], None if s["zeros"] is None else s["zeros"][of], s["cols"], s["group"])
        y = torch.bmm(w, x[:, :, None])[:, :, 0]
    else:  # all experts, each with as many rows as the fullest has
        w = _matrix(s["codes"], s["scales"], s["zeros"], s["cols"], s["group"])
        rows = (offsets[:-1, None] + torch.arange(s["most"], device=DEV)[None, :]).clamp(max=n - 1)
        y = torch.bmm(x[rows], w.transpose(1, 2))[of, i - offsets[of]]
    if s["op"] == "up":
        gate, up = y[:, 0::2], y[:, 1::2]
        y = gate / (1.0 + torch.exp(-gate)) * up
    s["y"].copy_(y)
    return s["y"]


def _plain_combine(s):
    rows = s["y"][s["slots"].long()].float()
    s["out"].copy_(s["residual"].float() + (rows * s["weights"][:, :, None]).sum(1))
    return s["out"]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        logit = s["logits"].double().cpu().numpy()
        best = np.argsort(-logit, axis=1, kind="stable")[:, :case["top_k"]]
        if case["score"] == "sigmoid":
            score = 1 / (1 + np.exp(-logit))
        else:
            score = np.exp(logit) / np.exp(logit).sum(1)[:, None]
        chosen = np.take_along_axis(score, best, 1)
        weights = chosen / chosen.sum(1)[:, None] if case["renorm"] else chosen
        return {"ids": None, "weights": torch.from_numpy(weights), "offsets": None, "order": None, "slots": None}
    if case["op"] == "combine":
        total = s["residual"].double()
        for j in range(case["top_k"]):
            total = total + s["weights"][:, j].double()[:, None] * s["y"].double().index_select(0, s["slots"][:, j].long())
        return total
    column = torch.arange(case["cols"], device=DEV)
    out = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    bounds = [0, case["tokens"]] if case["op"] == "linear" else s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if a == b:
            continue
        x = s["x"][s["order"][a:b].long() // case["top_k"]] if case["op"] == "up" else s["x"][a:b]
        codes, which = s["codes"][e].int(), column // case["group"]
        for r in range(0, case["rows"], 2048):
            part = slice(r, min(r + 2048, case["rows"]))
            code = codes[part][:, column // 2].bitwise_right_shift(4 * (column % 2).int()).remainder(16)
            zero = 8 if s["zeros"] is None else s["zeros"][e][part][:, which].int()
            y = torch.mm(x.double(), (s["scales"][e][part][:, which].double() * (code - zero).double()).t())
            if case["op"] == "up":
                out[a:b, r // 2:r // 2 + y.shape[1] // 2] = torch.special.expit(y[:, ::2]) * y[:, ::2] * y[:, 1::2]
            else:
                out[a:b, part] = y
    return out
