"""A NaN in a score that a row sees makes that row NaN, and no other row: in Q, in one key wherever it lies in its block,
its warp's or stream's piece and its unit's part, in both kernels of attention over a paged cache, whole and split.

Rows that see no NaN are held to cache_util.tolerance as everywhere; every column of the others is NaN.
"""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import DT, make_cache, pack_bits, run_attention, starts, tolerance, tree_bits, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def queries(seed, tokens, heads, dim, dtype):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((1.5 * rng.standard_normal((tokens, heads, dim))).astype(np.float32)).to(DT[dtype]).cuda()


def attention(q, k, v, ok, scale):
    """cache_util.attention64 for rows that all see something, a head at a time."""
    O, T, N, A = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), 0.0
    for h in range(q.shape[1]):
        kk, vv = (x[h // (q.shape[1] // k.shape[0])] for x in (k, v))
        s = np.where(ok, scale * (q[:, h] @ kk.T), -np.inf)
        p = np.exp(s - np.where(np.isnan(s), -np.inf, s).max(1, keepdims=True).clip(-1e300))
        p /= p.sum(1, keepdims=True)
        O[:, h], T[:, h], N[:, h] = p @ vv, p @ np.abs(vv), ok @ np.abs(vv)
        A = max(A, float(np.nan_to_num(np.where(ok, scale * (np.abs(q[:, h]) @ np.abs(kk).T), 0.0), nan=0.0).max()))
    return O, T, A, N


def check(c, dk, dv, q, counts, lens, window, sinks, dtype, bits=None, mask=None):
    """Returns how many (row, head)s are NaN."""
    scale = q.shape[2] ** -0.5
    got = run_attention(c, 0, q, counts, window, sinks, scale, mask=mask).double().cpu().numpy()
    qh, st, poisoned = q.double().cpu().numpy(), starts(counts), 0
    for s, n in enumerate(counts):
        a, e = st[s], st[s + 1]
        ok = visible(lens[s], n, window, sinks, None if bits is None else bits[s])
        O, T, A, N = attention(qh[a:e], dk[s][0], dv[s][0], ok, scale)
        want = np.isnan(O)
        assert np.array_equal(want.any(2), want.all(2))
        assert np.array_equal(np.isnan(got[a:e]), want), \
            f"sequence {s}: NaN where it should not be or not where it should, first at {np.argwhere(np.isnan(got[a:e]) != want)[0].tolist()}"
        clean = ~want
        assert (np.abs(got[a:e] - O)[clean] <= tolerance(T, N, A, q.shape[2], dtype)[clean]).all()
        poisoned += int(want.all(2).sum())
    return poisoned


def put(c, dk, s, j, head, value, column=3):
    """`value` into key j of sequence s, on the device and in the dense copy; returns what was there."""
    k, _, table, _, _ = c.tensors
    page = c.page_size
    row = k[0, int(table[s, j // page]), head, j % page]
    was = float(row[column])
    row[column] = value
    dk[s][0][head, j, column] = value
    return was


# (name, lens, new, heads, kv_heads, dim, page, window, sinks): units whole and split, rows kernel and tiles kernel
CASES = [
    ("one token", [16, 15, 100, 64], [1] * 4, 4, 2, 64, 16, 0, 0),
    ("one token, split", [5000], [1], 4, 2, 128, 64, 0, 0),
    ("one token, window", [900, 64], [1, 1], 4, 2, 64, 16, 65, 17),
    ("one token, the newest key alone in its part", [4096, 64, 128], [1] * 3, 2, 1, 64, 16, 0, 0),
    ("few rows", [64, 13], [3, 4], 4, 2, 64, 16, 0, 0),
    ("few rows, split", [3000], [4], 4, 1, 128, 32, 0, 0),
    ("40 rows", [0, 16, 90], [20, 20, 20], 4, 2, 64, 16, 0, 0),
    ("40 rows of 128, split", [2500], [20], 2, 1, 128, 64, 0, 0),
    ("40 rows, the second stream sees one key", [120, 119], [20, 20], 2, 1, 64, 16, 0, 0),
    ("128 rows on three blocks", [300], [64], 2, 1, 64, 16, 0, 0),
    ("300 rows", [70, 200], [150, 151], 2, 1, 64, 16, 0, 0),
    ("300 rows, split", [3000], [75], 4, 1, 128, 64, 0, 0),
    ("300 rows, window", [700], [150], 2, 1, 64, 16, 100, 17),
]
IDS = [c[0].replace(" ", "_").replace(",", "") for c in CASES]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_nan_in_one_key(case, dtype):
    _, lens, new, heads, kv_heads, dim, page, window, sinks = case
    c, dk, dv = make_cache(3, lens, new, kv_heads, dim, page, dtype)
    q = queries(5, sum(new), heads, dim, dtype)
    assert check(c, dk, dv, q, new, lens, window, sinks, dtype) == 0
    hit = 0
    for where in (0, 15, 16, 64, 127, 128, "first new", "newest", "middle"):
        at = []
        for s, (n, x) in enumerate(zip(lens, new)):
            j = {"first new": n, "newest": n + x - 1, "middle": (n + x) // 2}.get(where, where)
            if j < n + x:
                at.append((s, j, s % kv_heads))
        was = [put(c, dk, s, j, h, float("nan")) for s, j, h in at]
        hit += check(c, dk, dv, q, new, lens, window, sinks, dtype)
        for (s, j, h), w in zip(at, was):
            put(c, dk, s, j, h, w)
    assert hit > 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_nan_in_one_query(case, dtype):
    _, lens, new, heads, kv_heads, dim, page, window, sinks = case
    c, dk, dv = make_cache(4, lens, new, kv_heads, dim, page, dtype)
    q = queries(6, sum(new), heads, dim, dtype)
    for row, head in ((0, 0), (sum(new) - 1, heads - 1), (sum(new) // 2, heads // 2)):
        x = q.clone()
        x[row, head, dim - 1] = float("nan")
        assert check(c, dk, dv, x, new, lens, window, sinks, dtype) == 1


@pytest.mark.parametrize("n", [5, 16, 40, 150])
def test_nan_in_a_draft(n):
    # a drafted key that some rows see and others do not
    dtype, lens, rng = "bf16", [200, 31], np.random.default_rng(n)
    c, dk, dv = make_cache(8, lens, [n, n], 1, 64, 16, dtype)
    q = queries(7, 2 * n, 1, 64, dtype)
    bits = [tree_bits(rng, n), tree_bits(rng, n)]
    mask = pack_bits(np.concatenate(bits), -(-n // 32)).cuda()
    for t in (0, 1, n // 2, n - 1):
        was = [put(c, dk, s, lens[s] + t, 0, float("nan")) for s in range(2)]
        assert check(c, dk, dv, q, [n, n], lens, 0, 0, dtype, bits=bits, mask=mask) == int(bits[0][:, t].sum() + bits[1][:, t].sum())
        for s in range(2):
            put(c, dk, s, lens[s] + t, 0, was[s])
