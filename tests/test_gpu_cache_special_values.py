"""Infinities and NaN among the values of drafted and windowed tokens, which some rows see and others do not: every row has
what the definition gives it (NaN, plus or minus infinity where it sees them, the finite sum everywhere else), in both
kernels, whole and split, and at lengths where computing rows key by key would outlast the kernels' bounded waits.
"""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import DT, make_cache, pack_bits, run_attention, starts, tolerance, tree_bits, visible

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def expected(q, k, v, ok, scale):
    """O, T, N, A as cache_util.attention64 has them for rows that all see something, with the special values' part."""
    finite, nan, pos, neg = np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0), np.isnan(v), v == INF, v == -INF
    O, T, N, A = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), 0.0
    for h in range(q.shape[1]):
        g = h // (q.shape[1] // k.shape[0])
        s = np.where(ok, scale * (q[:, h] @ k[g].T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        O[:, h], T[:, h], N[:, h] = p @ finite[g], p @ np.abs(finite[g]), ok @ np.abs(finite[g])
        A = max(A, float(np.where(ok, scale * (np.abs(q[:, h]) @ np.abs(k[g]).T), 0.0).max()))
        sees = [(ok.astype(np.int64) @ x[g].astype(np.int64)) > 0 for x in (nan, pos, neg)]
        O[:, h][sees[1]] = INF
        O[:, h][sees[2]] = -INF
        O[:, h][sees[0] | (sees[1] & sees[2])] = NAN
    return O, T, N, A


def check(c, dk, dv, q, new, lens, window, sinks, dtype, bits=None, mask=None):
    scale = 0.05  # no weight near 0
    got = run_attention(c, 0, q, new, window, sinks, scale, mask=mask).double().cpu().numpy()
    qh, st, special = q.double().cpu().numpy(), starts(new), 0
    for s, n in enumerate(new):
        ok = visible(lens[s], n, window, sinks, None if bits is None else bits[s])
        O, T, N, A = expected(qh[st[s]:st[s + 1]], dk[s][0], dv[s][0], ok, scale)
        x = got[st[s]:st[s + 1]]
        odd = ~np.isfinite(O)
        assert np.array_equal(np.isnan(x), np.isnan(O)) and np.array_equal(x[odd & ~np.isnan(O)], O[odd & ~np.isnan(O)]), f"sequence {s}"
        assert (np.abs(x - np.where(odd, 0, O))[~odd] <= tolerance(T, N, A, q.shape[2], dtype)[~odd]).all(), f"sequence {s}"
        special += int(odd.sum())
    return special


def put(c, dv, s, j, head, column, value):
    _, v, table, _, _ = c.tensors
    v[0, int(table[s, j // c.page_size]), head, j % c.page_size, column] = value
    dv[s][0][head, j, column] = value


# (name, lens, new, heads, kv_heads, dim, page, window, sinks)
CASES = [
    ("few rows", [100, 31], [3, 4], 4, 2, 64, 16, 0, 0),
    ("few rows, window", [400, 77], [3, 1], 4, 2, 128, 16, 48, 5),
    ("few rows, split", [3000], [4], 4, 1, 64, 64, 0, 0),
    ("one tile", [100, 0], [40, 60], 4, 2, 64, 16, 0, 0),
    ("one tile, split", [2500], [30], 4, 1, 128, 64, 0, 0),
    ("two tiles", [300, 10], [130, 256], 4, 2, 128, 32, 0, 0),
    ("two tiles, window", [700], [150], 4, 2, 64, 16, 90, 17),
    ("two tiles, split", [2700], [60], 4, 1, 64, 64, 0, 0),
    ("many units", [50] * 40, [70] * 40, 8, 8, 64, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[c[0].replace(" ", "_").replace(",", "") for c in CASES])
def test_special_values(case, dtype):
    _, lens, new, heads, kv_heads, dim, page, window, sinks = case
    c, dk, dv = make_cache(3, lens, new, kv_heads, dim, page, dtype)
    rng = np.random.default_rng(5)
    q = torch.from_numpy(rng.standard_normal((sum(new), heads, dim)).astype(np.float32)).to(DT[dtype]).cuda()
    assert check(c, dk, dv, q, new, lens, window, sinks, dtype) == 0
    for s, (n, x) in enumerate(zip(lens, new)):
        edges = [n, n + x - 1, n + x // 2] + ([max(0, n - window), n - window + x, sinks - 1, sinks] if window else [0, n // 2])
        for i, j in enumerate(j for j in edges if 0 <= j < n + x):
            put(c, dv, s, j, s % kv_heads, (7 * i + s) % dim, (INF, -INF, NAN)[(i + s) % 3])
        put(c, dv, s, n, 0, dim - 1, INF)   # both infinities in a column: those that see both have NaN
        put(c, dv, s, n + x - 1, 0, dim - 1, -INF)
    assert check(c, dk, dv, q, new, lens, window, sinks, dtype) > 0
    s, n = 0, lens[0]
    for j in range(n, n + new[0]):  # and every new value of a head
        for d in range(dim):
            put(c, dv, s, j, 0, d, NAN)
    assert check(c, dk, dv, q, new, lens, window, sinks, dtype) > 0


@pytest.mark.parametrize("n,heads", [(6, 2), (60, 2), (300, 1)])
def test_special_values_in_a_tree(n, heads):
    dtype, lens, rng = "f16", [130, 40], np.random.default_rng(n)
    c, dk, dv = make_cache(8, lens, [n, n], 1, 64, 16, dtype)
    q = torch.from_numpy(rng.standard_normal((2 * n, heads, 64)).astype(np.float32)).half().cuda()
    bits = [tree_bits(rng, n), tree_bits(rng, n)]
    mask = pack_bits(np.concatenate(bits), -(-n // 32)).cuda()
    for s in range(2):
        for i, t in enumerate({0, 1, n // 2, n - 1}):
            put(c, dv, s, lens[s] + t, 0, 5 + i, (INF, NAN, -INF)[i % 3])
    assert check(c, dk, dv, q, [n, n], lens, 0, 0, dtype, bits=bits, mask=mask) > 0


def test_an_infinity_behind_a_long_context():
    # 160 sequences that share 250,000 tokens: more units than CTAs, so that a unit's end has others waiting behind it
    seqs, new, dim, page, n = 160, 256, 64, 128, 250_000
    held = -(-(n + new) // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, held, 1, page, dim), generator=g, device="cuda").half() for _ in range(2))
    table = torch.arange(held, dtype=torch.int32, device="cuda").repeat(seqs, 1).contiguous()
    c = mm.mm_cache(k, v, table, torch.full((seqs,), n, dtype=torch.int32, device="cuda"))
    q = torch.randn((seqs * new, 1, dim), generator=g, device="cuda").half()
    v[0, (n + 3) // page, 0, (n + 3) % page, 5] = 0
    clean = run_attention(c, 0, q, [new] * seqs, 0, 0, 0.05)
    v[0, (n + 3) // page, 0, (n + 3) % page, 5] = INF
    got = run_attention(c, 0, q, [new] * seqs, 0, 0, 0.05).view(seqs, new, dim)
    clean = clean.view(seqs, new, dim)
    assert bool((got[:, 3:, 5] == INF).all())
    got[:, 3:, 5] = clean[:, 3:, 5]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))
