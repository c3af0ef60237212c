"""A paged cache for the tests, and attention over it written from its definition in fp64 (CPU).

Everything that no token occupies -- pages nobody holds, the rest of each last page -- is NaN, and
so is what lies between the rows of a strided tensor: an access that should not matter shows.
"""
import numpy as np
import torch

import dense_packed_bit_gb300 as mm

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # largest relative error of one rounding


def make_cache(seed, lens, extra, kv_heads, dim, page, dtype, layers=1, spare=3, max_pages=None, device="cuda",
               layout="heads", dense=None):
    """lens[s] committed tokens and extra[s] new ones per sequence, in pages of random numbers.
    layout: "heads" [page][head][token], "tokens" [page][token][head], "padded" rows padded to a wider
    stride, "both" K and V interleaved in one allocation.  Returns (cache, dense k, dense v): dense is
    per layer and sequence [kv_heads][tokens][dim] float64 on the CPU."""
    rng = np.random.default_rng(seed)
    total = [a + b for a, b in zip(lens, extra)]
    held = [-(-t // page) for t in total]
    max_pages = max_pages or max(held + [1]) + 1
    pages = sum(held) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max_pages), -1, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    at = 0
    for s, h in enumerate(held):
        table[s, :h] = order[at:at + h]
        refs[order[at:at + h]] = 1
        at += h
    dt = DT[dtype]
    data = [[rng.standard_normal((layers, kv_heads, t, dim)).astype(np.float32) for t in total] for _ in range(2)]
    pool = torch.full((2, layers, pages, kv_heads, page, dim), float("nan"), dtype=dt)
    dense_out = []
    for w in range(2):
        dense_w = []
        for s, t in enumerate(total):
            d = torch.from_numpy(data[w][s]).to(dt)
            dense_w.append(d.double().numpy())
            for j in range(0, t, page):
                n = min(page, t - j)
                pool[w, :, table[s, j // page], :, :n] = d[:, :, j:j + n]
        dense_out.append(dense_w)
    if layout == "tokens":
        pool = pool.permute(0, 1, 2, 4, 3, 5).contiguous().to(device).permute(0, 1, 2, 4, 3, 5)
        k, v = pool[0], pool[1]
    elif layout == "padded":
        wide = torch.full((2, layers, pages, kv_heads, page, dim + 24), float("nan"), dtype=dt)
        wide[..., 8:8 + dim] = pool
        wide = wide.to(device)
        k, v = wide[0, ..., 8:8 + dim], wide[1, ..., 8:8 + dim]
    elif layout == "both":
        both = pool.permute(1, 2, 0, 3, 4, 5).contiguous().to(device)  # [layers][pages][2]...
        k, v = both[:, :, 0], both[:, :, 1]
    else:
        pool = pool.to(device)
        k, v = pool[0], pool[1]
    c = mm.mm_cache(k, v, torch.from_numpy(table).to(device), torch.tensor(lens, dtype=torch.int32, device=device),
                    torch.from_numpy(refs).to(device))
    return c, dense_out[0], dense_out[1]


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def visible(n, count, window, sinks, bits=None):
    """[count][n + count] truth values; bits: [count][count] of the tree, or None (causal)."""
    j = np.arange(n + count)[None, :]
    if bits is None:
        p = n + np.arange(count)[:, None]
        ok = j <= p
        drafted = np.zeros_like(ok)
    else:
        p = n + bits.sum(1, keepdims=True) - 1
        drafted = j >= n
        ok = np.concatenate([np.ones((count, n), dtype=bool), bits], 1)
    if window:
        ok = ok & ((j > p - window) | (j < sinks) | (drafted & (j >= n)))
    return ok


def attention64(q, k, v, ok, scale):
    """(O, T, A, N): q [count][heads][dim], k, v [kv_heads][keys][dim], fp64; T = sum p |v| over the visible
    keys, A = the largest sum |q k| scale, N = sum |v| over the visible keys.  Masked places are not touched."""
    count, heads, dim = q.shape
    group = heads // k.shape[0]
    O, T, N = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    A = 0.0
    for h in range(heads):
        kk, vv = k[h // group], v[h // group]
        for i in range(count):
            at = np.flatnonzero(ok[i])
            if at.size == 0:
                continue
            s = scale * (kk[at] @ q[i, h])
            A = max(A, float(np.max(scale * (np.abs(kk[at]) @ np.abs(q[i, h])))))
            p = np.exp(s - s.max())
            p /= p.sum()
            O[i, h], T[i, h], N[i, h] = p @ vv[at], p @ np.abs(vv[at]), np.abs(vv[at]).sum(0)
    return O, T, A, N


def tolerance(T, N, A, dim, dtype):
    """Probabilities and O each rounded once to the cache's type (u T each, with fp16's subnormal step below
    that), scores as fp32 sums of dim products (passed on at most twice), exp2 and the sums 1e-5."""
    u = UNIT[dtype]
    sub = 2.0 ** -25 if dtype == "f16" else 2.0 ** -133
    return (2 * u * (1 + u) + 1e-5 + 4 * dim * 2.0 ** -24 * A) * T + sub * (1 + N)


def run_attention(c, layer, q, counts, window, sinks, scale, mask=None, max_q=None, ws=None, stream=None, pad=0):
    """q: [tokens][heads][dim] device tensor; O comes back between guard rows, all of it checked."""
    tokens, heads, dim = q.shape
    qs = torch.from_numpy(starts(counts)).to(q.device)
    guard = 2
    buf = torch.full((tokens + 2 * guard, heads * dim + pad), 7.0, dtype=q.dtype, device=q.device)
    out = buf[guard:guard + tokens, :heads * dim].view(tokens, heads, dim) if pad == 0 else \
        buf[guard:guard + tokens, :heads * dim].unflatten(1, (heads, dim))
    max_q = max_q or max(counts)
    if ws is None:
        ws = torch.zeros(max(mm.mm_cache_attention_workspace(c, heads, tokens, max_q), 16), dtype=torch.uint8,
                         device=q.device)
    if mask is None:
        mm.mm_cache_attention(c, layer, q, q.stride(0), heads, qs, tokens, max_q, window, sinks, scale, out,
                              out.stride(0), ws, ws.numel(), stream)
    else:
        mm.mm_cache_attention_tree(c, layer, q, q.stride(0), heads, qs, tokens, max_q, mask, mask.shape[1], window,
                                   sinks, scale, out, out.stride(0), ws, ws.numel(), stream)
    torch.cuda.synchronize()
    mm.mm_check_device_error()
    assert bool((buf[:guard] == 7).all()) and bool((buf[guard + tokens:] == 7).all()), "rows around O written"
    if pad:
        assert bool((buf[:, heads * dim:] == 7).all()), "columns past O written"
    return out


def pack_bits(rows, words):
    """Truth values [tokens][n] as [tokens][words] int32."""
    out = np.zeros((rows.shape[0], words), dtype=np.uint32)
    for t in range(rows.shape[1]):
        out[:, t // 32] |= rows[:, t].astype(np.uint32) << np.uint32(t % 32)
    return torch.from_numpy(out.view(np.int32))


def tree_bits(rng, n):
    """A random tree of n drafts: [n][n], each sees itself and its ancestors."""
    bits = np.zeros((n, n), dtype=bool)
    for i in range(n):
        if i and rng.random() < 0.85:
            bits[i] = bits[rng.integers(0, i)]
        bits[i, i] = True
    return bits


def check_attention(c, dk, dv, layer, q, counts, lens, window, sinks, scale, dtype, bits=None, out=None, mask=None,
                    **kw):
    if out is None:
        out = run_attention(c, layer, q, counts, window, sinks, scale, mask=mask, **kw)
    got, qh, st = out.double().cpu().numpy(), q.double().cpu().numpy(), starts(counts)
    worst = 0.0
    for s, n in enumerate(counts):
        if n == 0:
            continue
        a, e = st[s], st[s + 1]
        ok = visible(lens[s], n, window, sinks, None if bits is None else bits[s])
        O, T, A, N = attention64(qh[a:e], dk[s][layer], dv[s][layer], ok, scale)
        tol = tolerance(T, N, A, q.shape[2], dtype)
        assert np.all(np.isfinite(got[a:e])), f"sequence {s}: not finite"
        off = np.abs(got[a:e] - O)
        bad = off > tol
        assert not bad.any(), (f"sequence {s}: {int(bad.sum())} of {bad.size} outside, worst {float((off / np.maximum(tol, 1e-300)).max()):.2f} "
                               f"times the tolerance at {np.argwhere(bad)[0].tolist()}")
        worst = max(worst, float((off / np.maximum(tol, 1e-300)).max()))
    return worst, out
