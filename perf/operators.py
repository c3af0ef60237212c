"""What is measured of the operators that serve a language model's tokens from a paged cache of keys and values.

Four of them, as a server runs them between the packed products of a step:

  attention  the new tokens of a ragged batch (one token each, or a chunk of a prompt) against the cache, with
             a sliding window and a few first tokens that stay visible
  tree       a tree of drafted tokens per sequence against the cache, each seeing the cached tokens and its ancestors
  sample     the next token of each row of logits by temperature, top-k, top-p and min-p from given random numbers
  pages      the cache's bookkeeping: forking sequences (shared full pages, a copied last page), and a round of
             drafted tokens (pages reserved, tokens written, the accepted ones moved together, the rest released)

A cache is k, v [layers][pages][kv heads][page size][head dim], table [sequences][max pages], lens [sequences]
and refs [pages] (how many sequences hold a page).  `lens` counts the tokens that stay; the new (or drafted) tokens
of sequence s follow them, at positions lens[s] + i, and are rows q_start[s] .. q_start[s + 1] of Q.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLOATS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FIXED = 1 << 30  # a token's weight is held in 30 fractional bits of the row's largest


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one sequence, one token: GPT-2's heads early in an answer; a latency
        dict(name="decode 1 x 513", op="attention", seqs=1, lo=513, hi=513, new_lo=1, new_hi=1, heads=12, kv_heads=12,
             dim=64, page=16, window=0, sinks=0, dtype="f16"),
        # a server's full batch of ragged answers, grouped heads: reading the cache is all of it
        dict(name="decode 48 ragged", op="attention", seqs=48, lo=100, hi=16000, new_lo=1, new_hi=1, heads=32,
             kv_heads=8, dim=128, page=64, window=0, sinks=0, dtype="bf16"),
        # long answers under a window: a few pages of many are read (1,536-wide rows: 12 heads of 128)
        dict(name="decode 8 window of 32k", op="attention", seqs=8, lo=30011, hi=32700, new_lo=1, new_hi=1, heads=12,
             kv_heads=2, dim=128, page=32, window=1024, sinks=4, dtype="f16"),
        # chunks of several prompts, GPT-2's heads, ragged in what is new and in what is cached
        dict(name="prefill 4 ragged", op="attention", seqs=4, lo=1, hi=700, new_lo=150, new_hi=1024, heads=12,
             kv_heads=12, dim=64, page=16, window=0, sinks=0, dtype="f16"),
        # a chunk of a long document under a window: the matrix products bound it
        dict(name="prefill 4096 on 12k", op="attention", seqs=1, lo=12289, hi=12289, new_lo=4096, new_hi=4096, heads=32,
             kv_heads=8, dim=128, page=64, window=4096, sinks=64, dtype="bf16"),
        # small trees of a few sequences
        dict(name="tree 4 x 7", op="tree", seqs=4, lo=300, hi=1100, new_lo=7, new_hi=7, heads=12, kv_heads=12, dim=64,
             page=16, window=0, sinks=0, dtype="f16"),
        # wide trees of a batch over long answers
        dict(name="tree 16 x 64", op="tree", seqs=16, lo=2500, hi=8000, new_lo=64, new_hi=64, heads=32, kv_heads=8,
             dim=128, page=64, window=0, sinks=0, dtype="bf16"),
        # one row of GPT-2's vocabulary: a latency
        dict(name="sample 1 x 50257", op="sample", rows=1, vocab=50257, dtype="f32"),
        # a batch's step in 16 bits
        dict(name="sample 64 x 50257", op="sample", rows=64, vocab=50257, dtype="bf16"),
        # many rows of a large vocabulary: reading the logits
        dict(name="sample 512 x 128000", op="sample", rows=512, vocab=128000, dtype="f32"),
        # every answer of a batch forked eight ways, all layers' last pages copied
        dict(name="fork 8 into 64", op="fork", parents=8, children=64, layers=16, lo=900, hi=4000, kv_heads=8, dim=128,
             page=64, dtype="bf16"),
        # a verification round of small trees
        dict(name="round 16 x 12", op="round", seqs=16, lo=200, hi=1000, draft=12, layers=1, kv_heads=12, dim=64,
             page=16, dtype="f16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "tree", "sample", "sample", "fork", "round"])
    if op == "sample":
        vocab = _log(rng, 1000, 128000)
        return dict(op="sample", rows=_log(rng, 1, 512), vocab=vocab, dtype=rng.choice(["f16", "bf16", "f32"]))
    kv_heads, group, dim = rng.choice([(12, 1, 64), (8, 4, 128), (2, 6, 128), (4, 2, 64), (1, 8, 128), (5, 3, 80), (2, 7, 96)])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    if op == "fork":
        parents = _log(rng, 1, 8)
        lo = _log(rng, 20, 2000)
        return dict(op="fork", parents=parents, children=parents * _log(rng, 1, 8), layers=_log(rng, 1, 8), lo=lo,
                    hi=2 * lo, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)
    if op == "round":
        lo = _log(rng, 20, 2000)
        return dict(op="round", seqs=_log(rng, 1, 48), lo=lo, hi=2 * lo, draft=_log(rng, 2, 64), layers=1,
                    kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)
    window = rng.choice([0, 0, _log(rng, 64, 4096)])
    sinks = rng.choice([0, 4, 64]) if window else 0
    case = dict(op="tree" if op == "tree" else "attention", heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                page=page, window=window, sinks=sinks, dtype=dtype)
    if op == "decode":
        lo = _log(rng, 50, 1500)
        return dict(case, seqs=_log(rng, 1, 32), lo=lo, hi=_log(rng, lo, 8000), new_lo=1, new_hi=1)
    if op == "tree":
        lo = _log(rng, 50, 3000)
        new = _log(rng, 2, 64)
        return dict(case, seqs=_log(rng, 1, 16), lo=lo, hi=2 * lo, new_lo=new, new_hi=new)
    seqs, hi = _log(rng, 1, 4), _log(rng, 64, 2048)
    return dict(case, seqs=seqs, lo=1, hi=_log(rng, 2, 2500), new_lo=max(1, hi // 3), new_hi=hi)


# ------------------------------------------------------------------ sizes that go by the case alone

def _spread(n, lo, hi, shift):
    """n whole numbers over lo .. hi, spread evenly over their logarithm, in a scattered order."""
    t = (np.arange(n) * 0.6180339887 + shift) % 1.0
    return np.clip(np.round(lo * (hi / lo) ** t), lo, hi).astype(np.int64)


def _lengths(case):
    """(cached tokens, new tokens) of each sequence."""
    if case["op"] == "round":
        return _spread(case["seqs"], case["lo"], case["hi"], 0.37), np.full(case["seqs"], case["draft"], dtype=np.int64)
    return (_spread(case["seqs"], case["lo"], case["hi"], 0.37),
            _spread(case["seqs"], case["new_lo"], case["new_hi"], 0.81))


def _tree(n):
    """Parents of a draft tree of n tokens: -1 is the last cached token; up to three branches at each token."""
    parent = np.full(n, -1, dtype=np.int64)
    for i in range(1, n):
        parent[i] = (i - 1) // 3 if i % 4 else i - 1
    return parent


def _ancestors(n):
    """seen[i][j]: whether drafted token i sees drafted token j (itself and its ancestors)."""
    parent, seen = _tree(n), np.zeros((n, n), dtype=bool)
    for i in range(n):
        if parent[i] >= 0:
            seen[i] = seen[parent[i]]
        seen[i, i] = True
    return seen


def _kept(case):
    """How many of a round's drafted tokens are accepted, per sequence."""
    return np.minimum(_spread(case["seqs"], 1, case["draft"], 0.11), case["draft"])


def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * 28, "flops": 4 * n}
    row = case["kv_heads"] * case["dim"] * size
    if case["op"] == "fork":
        part = _spread(case["parents"], case["lo"], case["hi"], 0.37) % case["page"]
        moved = int(part[np.arange(case["children"]) % case["parents"]].sum())
        return {"bytes": 4 * case["layers"] * row * moved + 8 * case["children"], "flops": 0}
    if case["op"] == "round":
        new, kept = case["seqs"] * case["draft"], int(_kept(case).sum())
        return {"bytes": 4 * case["layers"] * row * (new + kept) + 8 * new, "flops": 0}
    cached, new = _lengths(case)
    read = pairs = 0
    for n, q in zip(cached.tolist(), new.tolist()):
        if case["op"] == "tree":
            seen = _ancestors(q)
            at, own_seen = n + seen.sum(1) - 1, seen.sum(1)
        else:
            at, own_seen = n + np.arange(q), None
        low = np.maximum(0, at - case["window"] + 1) if case["window"] else np.zeros(q, dtype=np.int64)
        first = np.minimum(low, case["sinks"])
        if own_seen is None:
            pairs += int((at + 1 - low + first).sum())
        else:
            pairs += int((np.maximum(0, n - low) + np.minimum(first, n) + own_seen).sum())
        read += int(n + q - low.min() + first.min())
    io = 2 * int(new.sum()) * case["heads"] * case["dim"] * size
    return {"bytes": 2 * row * read + io, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ what a program has in hand

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)

    def ints(a):
        return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)

    dtype = FLOATS[case["dtype"]]
    if case["op"] == "sample":
        n = case["rows"]

        def uniform(lo, hi):
            return lo + (hi - lo) * torch.rand(n, generator=g, device=DEV)

        return dict(op="sample", logits=normal(n, case["vocab"], dtype=dtype, scale=3.0), temperature=uniform(0.5, 1.2),
                    top_k=torch.randint(20, 200, (n,), generator=g, device=DEV, dtype=torch.int32),
                    top_p=uniform(0.8, 1.0), min_p=uniform(0.0, 0.05),
                    u=torch.rand(n, generator=g, device=DEV),
                    tokens=torch.empty(n, dtype=torch.int32, device=DEV),
                    logprobs=torch.empty(n, dtype=torch.float32, device=DEV))
    page, dim, kv_heads = case["page"], case["dim"], case["kv_heads"]
    if case["op"] == "fork":
        parents, children = case["parents"], case["children"]
        lens = np.concatenate([_spread(parents, case["lo"], case["hi"], 0.37), np.zeros(children, dtype=np.int64)])
        width = -(-case["hi"] // page) + 1
        held, spare = -(-lens // page), children + 2
    else:
        lens, new = _lengths(case)
        width = -(-int((lens + new).max()) // page)
        held, spare = -(-(lens if case["op"] == "round" else lens + new) // page), 0
        if case["op"] == "round":
            spare = int((-(-(lens + new) // page) - held).sum()) + 3
    seqs, used = len(lens), int(held.sum())
    pages, layers = used + spare, case.get("layers", 1)
    order = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    holds = np.arange(width)[None, :] < held[:, None]
    place = np.cumsum(holds).reshape(holds.shape) - 1
    table = torch.where(torch.as_tensor(holds).to(DEV), order[torch.as_tensor(np.maximum(place, 0)).to(DEV)], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order.long()] = 1
    shape = (layers, pages, kv_heads, page, dim)
    state = dict(op=case["op"], k=normal(*shape, dtype=dtype), v=normal(*shape, dtype=dtype), table=table.contiguous(),
                 lens=ints(lens), refs=refs)
    if case["op"] == "fork":
        return dict(state, parents=ints(np.arange(children) % parents), children=ints(parents + np.arange(children)),
                    missing=torch.zeros(1, dtype=torch.int32, device=DEV))
    starts = np.concatenate([[0], np.cumsum(new)])
    state |= dict(q_start=ints(starts), tokens=int(starts[-1]), max_q=int(new.max()))
    if case["op"] == "round":
        kept, n = _kept(case), case["draft"]
        pick = torch.rand(seqs, n, generator=g, device=DEV).argsort(1).to(torch.int32)
        inside = torch.arange(n, device=DEV)[None, :] < torch.as_tensor(kept).to(DEV)[:, None]
        keep = torch.where(inside, pick, n).sort(1).values.clamp(max=n - 1)
        return dict(state, lens0=ints(lens), need=ints(new), kept=ints(kept), keep=keep.reshape(-1).to(torch.int32).contiguous(),
                    k_new=normal(state["tokens"], kv_heads, dim, dtype=dtype), v_new=normal(state["tokens"], kv_heads, dim, dtype=dtype),
                    missing=torch.zeros(1, dtype=torch.int32, device=DEV))
    q = normal(state["tokens"], case["heads"], dim, dtype=dtype, scale=1.5)
    state |= dict(q=q, out=torch.empty_like(q), window=case["window"], sinks=case["sinks"], scale=1.0 / math.sqrt(dim))
    if case["op"] == "tree":
        n = int(new.max())
        words = -(-n // 32)
        bits = np.zeros((state["tokens"], words), dtype=np.uint32)
        for s, c in enumerate(new.tolist()):
            i, j = np.nonzero(_ancestors(c))
            np.bitwise_or.at(bits, (starts[s] + i, j // 32), (np.uint32(1) << (j % 32).astype(np.uint32)))
        state |= dict(mask=torch.from_numpy(bits.view(np.int32)).to(DEV), words=words)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "tree": _plain_attention, "sample": _plain_sample, "fork": _plain_fork,
            "round": _plain_round}[state["op"]](state)


def _own(s):
    import dense_packed_bit_gb300 as mm
    if s["op"] == "sample":
        mm.mm_sample(s["logits"], s["logits"].shape[0], s["logits"].shape[1], s["logits"].stride(0), s["temperature"],
                     s["top_k"], s["top_p"], s["min_p"], s["u"], s["tokens"], s["logprobs"])
        return {"tokens": s["tokens"], "logprobs": s["logprobs"]}
    c = s.get("cache")
    if c is None:
        c = s["cache"] = mm.mm_cache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    if s["op"] == "fork":
        n = s["children"].shape[0]
        mm.mm_cache_free(c, s["children"], n, 0, 0)
        mm.mm_cache_fork(c, s["parents"], s["children"], n, s["missing"])
        return {x: s[x] for x in ("k", "v", "table", "lens", "refs", "missing")}
    if s["op"] == "round":
        s["lens"].copy_(s["lens0"])
        mm.mm_cache_reserve(c, s["need"], s["missing"])
        mm.mm_cache_append(c, 0, s["k_new"], s["v_new"], s["k_new"].stride(0), s["q_start"], s["tokens"], s["max_q"])
        mm.mm_cache_compact(c, s["q_start"], s["keep"], s["kept"], s["tokens"], s["max_q"])
        return {x: s[x] for x in ("k", "v", "table", "lens", "refs", "missing")}
    q, out = s["q"], s["out"]
    ws = s.get("workspace")
    if ws is None:
        n = mm.mm_cache_attention_workspace(c, q.shape[1], s["tokens"], s["max_q"])
        ws = s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    if s["op"] == "tree":
        mm.mm_cache_attention_tree(c, 0, q, q.stride(0), q.shape[1], s["q_start"], s["tokens"], s["max_q"], s["mask"],
                                   s["words"], s["window"], s["sinks"], s["scale"], out, out.stride(0), ws, ws.numel())
    else:
        mm.mm_cache_attention(c, 0, q, q.stride(0), q.shape[1], s["q_start"], s["tokens"], s["max_q"], s["window"],
                              s["sinks"], s["scale"], out, out.stride(0), ws, ws.numel())
    return out


def _plain_attention(s):
    q, q_start, lens, n = s["q"], s["q_start"].long(), s["lens"].long(), s["tokens"]
    k, v, table = s["k"][0], s["v"][0], s["table"].long().clamp(min=0)
    seqs, width = table.shape
    kv_heads, page, dim = k.shape[1:]
    heads, mq = q.shape[1], s["max_q"]
    keys = width * page
    i = torch.arange(mq, device=q.device)
    count = q_start[1:] - q_start[:-1]
    rows = (q_start[:-1, None] + i[None, :]).clamp(max=n - 1)
    qs = q[rows].float().view(seqs, mq, kv_heads, heads // kv_heads, dim).permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, -1, dim)
    ks = k[table].float().permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, keys, dim)
    vs = v[table].float().permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, keys, dim)
    j = torch.arange(keys, device=q.device)[None, None, :]
    if "mask" in s:
        words = s["mask"].long()[rows]                                                # [seqs][mq][words]
        bits = (words[..., None] >> torch.arange(32, device=q.device)) & 1
        bits = bits.reshape(seqs, mq, -1)
        at = lens[:, None] + bits.sum(-1) - 1
        d = j - lens[:, None, None]
        drafted = (d >= 0) & (d < count[:, None, None])
        bit = bits.gather(2, d.clamp(0, bits.shape[2] - 1).expand(seqs, mq, keys)).bool()
        seen = torch.where(drafted, bit, d < 0)
    else:
        at = lens[:, None] + i[None, :]
        drafted = torch.zeros((), dtype=torch.bool, device=q.device)
        seen = j <= at[..., None]
    if s["window"]:
        seen = seen & ((j > at[..., None] - s["window"]) | (j < s["sinks"]) | drafted)
    seen = seen[:, None, :, None, :].expand(seqs, 1, mq, heads // kv_heads, keys).reshape(seqs, 1, -1, keys)
    score = torch.matmul(qs, ks.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    out = torch.matmul(p, vs) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.view(seqs, kv_heads, mq, heads // kv_heads, dim).permute(0, 2, 1, 3, 4).reshape(seqs, mq, heads, dim)
    t = torch.arange(n, device=q.device)
    of = torch.searchsorted(q_start, t, right=True) - 1
    return out[of, t - q_start[of]].to(q.dtype)


def _plain_sample(s):
    x = s["logits"].float()
    x = x.masked_fill(torch.isnan(x), -math.inf)
    m = x.amax(1, keepdim=True)
    rate = (1.0 / s["temperature"].clamp(min=0))[:, None]
    z = torch.where(x == m, 0.0, (x - m) * rate).masked_fill(x == -math.inf, -math.inf)
    w = torch.round(torch.exp(z) * FIXED).long()
    k = torch.where(s["temperature"] > 0, s["top_k"], 1).long()
    k = torch.where(k > 0, k, w.shape[1])[:, None]
    order = w.sort(dim=1, descending=True, stable=True)
    rank = torch.arange(w.shape[1], device=w.device)[None, :]
    ranked = torch.where(rank < k, order.values, 0)
    mass = ranked.sum(1, keepdim=True)
    reached = ranked.cumsum(1) - ranked                                             # the mass before each
    target = torch.ceil(s["top_p"].double()[:, None] * mass.double()).long()
    inside = (rank == 0) | (reached < target)
    inside &= ranked >= torch.ceil(s["min_p"] * float(FIXED)).long()[:, None]
    keep = torch.zeros_like(w).scatter(1, order.indices, torch.where(inside, ranked, 0))
    total = keep.sum(1, keepdim=True)
    want = torch.floor(s["u"].double()[:, None] * total.double()).long()
    token = (keep.cumsum(1) <= want).sum(1)
    chosen = keep.gather(1, token.clamp(max=w.shape[1] - 1)[:, None])
    logprob = -torch.log1p((total - chosen).float() / chosen.float())[:, 0]
    none = total[:, 0] == 0
    return {"tokens": torch.where(none, -1, token).int(), "logprobs": torch.where(none, -math.inf, logprob)}


def _release(refs, rows, which):
    refs.scatter_add_(0, torch.where(which, rows, 0).reshape(-1).long(), -which.reshape(-1).int())


def _plain_fork(s):
    k, v, table, lens, refs = (s[x] for x in ("k", "v", "table", "lens", "refs"))
    parents, children = s["parents"].long(), s["children"].long()
    page, width = k.shape[3], table.shape[1]
    rows = table[children]
    _release(refs, rows, rows >= 0)
    n = lens[parents].long()
    full, part = n // page, n % page
    need = part > 0
    free = (refs != 0).sort(stable=True).indices
    lacking = (need.sum() - (refs == 0).sum()).clamp(min=0)
    ok = lacking == 0
    source = table[parents]
    last = source.gather(1, full.clamp(max=width - 1)[:, None])[:, 0].long()
    fresh = free[(need.cumsum(0) - 1).clamp(0, refs.shape[0] - 1)]
    col = torch.arange(width, device=k.device)[None, :]
    shared = (col < full[:, None]) & ok
    tail = (col == full[:, None]) & need[:, None] & ok
    table[children] = torch.where(shared, source, torch.where(tail, fresh[:, None].int(), -1)).int()
    refs.scatter_add_(0, torch.where(shared, source, 0).reshape(-1).long(), shared.reshape(-1).int())
    refs.scatter_add_(0, fresh, (need & ok).int())
    lens[children] = torch.where(ok, n, 0).int()
    copied = need & ok
    to = torch.where(copied, fresh, last.clamp(min=0))
    here = (torch.arange(page, device=k.device)[None, :] < part[:, None])[None, :, None, :, None] & copied[None, :, None, None, None]
    k[:, to] = torch.where(here, k[:, last.clamp(min=0)], k[:, to])
    v[:, to] = torch.where(here, v[:, last.clamp(min=0)], v[:, to])
    s["missing"].copy_(lacking)
    return {x: s[x] for x in ("k", "v", "table", "lens", "refs", "missing")}


def _plain_round(s):
    k, v, table, lens, refs, q_start = (s[x] for x in ("k", "v", "table", "lens", "refs", "q_start"))
    page, width, n = k.shape[3], table.shape[1], s["tokens"]
    lens.copy_(s["lens0"])
    col = torch.arange(width, device=k.device)[None, :]
    # pages for the drafted tokens: the lowest free ones, in the order of the sequences
    upto = (lens + s["need"] + page - 1) // page
    need = (col < upto[:, None]) & (table < 0)
    lacking = (need.sum() - (refs == 0).sum()).clamp(min=0)
    need = need & (lacking == 0)
    free = (refs != 0).sort(stable=True).indices
    fresh = free[(need.reshape(-1).cumsum(0) - 1).clamp(0, refs.shape[0] - 1)].view_as(table)
    table.copy_(torch.where(need, fresh.int(), table))
    refs.scatter_add_(0, fresh.reshape(-1), need.reshape(-1).int())
    s["missing"].copy_(lacking)
    # the drafted tokens into their slots
    t = torch.arange(n, device=k.device)
    of = torch.searchsorted(q_start.long(), t, right=True) - 1
    at = lens[of].long() + t - q_start[of].long()
    k[0][table[of, at // page].long(), :, at % page] = s["k_new"]
    v[0][table[of, at // page].long(), :, at % page] = s["v_new"]
    # the accepted ones together
    i = t - q_start[of].long()
    stays = i < s["kept"][of]
    source = lens[of].long() + torch.where(stays, s["keep"].long(), i)
    from_page, to_page = table[of, source // page].long(), table[of, at // page].long()
    k[:, to_page, :, at % page] = k[:, from_page, :, source % page]
    v[:, to_page, :, at % page] = v[:, from_page, :, source % page]
    # and the pages behind them back
    lens += s["kept"]
    beyond = (col >= ((lens + page - 1) // page)[:, None]) & (table >= 0)
    _release(refs, table, beyond)
    table.masked_fill_(beyond, -1)
    return {x: s[x] for x in ("k", "v", "table", "lens", "refs", "missing")}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] in ("fork", "round"):
        return None  # whole values and copies only: nothing is computed in floating point
    s = prepare(case, seed)
    if case["op"] == "sample":
        if case["rows"] * case["vocab"] > 8_000_000:
            return None
        return {"tokens": None, "logprobs": _exact_logprobs(s)}
    q_start, lens = s["q_start"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = case["heads"] // case["kv_heads"]
    for b in range(case["seqs"]):
        a, e = q_start[b], q_start[b + 1]
        total = lens[b] + e - a
        index = torch.arange(total, device=DEV)
        page = s["table"][b].long()[index // case["page"]]
        pos = torch.arange(a, e, device=DEV) - a
        if case["op"] == "tree":
            tree = torch.from_numpy(_ancestors(e - a)).to(DEV)
            allowed = torch.cat([torch.ones(e - a, lens[b], dtype=torch.bool, device=DEV), tree], 1)
            depth = lens[b] + tree.sum(1) - 1
        else:
            depth = lens[b] + pos
            allowed = index[None, :] <= depth[:, None]
        if case["window"]:
            near = (depth[:, None] - index[None, :] < case["window"]) | (index < case["sinks"])[None, :]
            if case["op"] == "tree":
                near[:, lens[b]:] = True
            allowed = allowed & near
        for h in range(case["kv_heads"]):
            key = s["k"][0, page, h, index % case["page"]].double()
            value = s["v"][0, page, h, index % case["page"]].double()
            for head in range(h * group, (h + 1) * group):
                logit = s["scale"] * (s["q"][a:e, head].double() @ key.T)
                weight = torch.softmax(torch.where(allowed, logit, -math.inf), dim=1)
                out[a:e, head] = weight @ value
    return out


def _exact_logprobs(s):
    """Row by row on the host: the weights by numpy in 64 bits, the filters one after another."""
    found = []
    logits = s["logits"].double().cpu().numpy()
    params = [s[x].double().cpu().numpy() for x in ("temperature", "top_k", "top_p", "min_p", "u")]
    for x, temperature, top_k, top_p, min_p, u in zip(logits, *params):
        w = np.rint(np.exp((x - x.max()) / temperature) * FIXED).astype(np.int64)
        order = np.lexsort((np.arange(w.size), -w))[: int(top_k) if top_k > 0 else w.size]
        sums = np.cumsum(w[order])
        count = int(np.searchsorted(sums, math.ceil(top_p * sums[-1]), side="left")) + 1
        order = order[:count]
        order = np.sort(order[w[order] >= min_p * FIXED])
        sums = np.cumsum(w[order])
        at = int(np.searchsorted(sums, math.floor(u * int(sums[-1])), side="right"))
        found.append(math.log(int(w[order[at]])) - math.log(int(sums[-1])))
    return torch.tensor(found, dtype=torch.float64)
