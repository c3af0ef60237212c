"""Sampling on the GPU (mm_sample) against its definition row by row in numpy.

Weights are whole numbers, so tokens are compared for equality.  The definition's exp is fp32; numpy's and
the GPU's may differ in the last bit, so a row where any decision lies within that of its bound (the cut of
top-p, of min-p, the token itself) accepts the tokens of both sides; log-probabilities follow the token.
"""
import math

import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm

pytestmark = pytest.mark.gpu

ONE = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def weights(x, temperature):
    """Weights by the definition, and how far fp32 may be off in each: exp's last bits, the products' in z."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    m = x.max() if x.size else -np.inf
    if m == -np.inf:
        return np.zeros(x.size, dtype=np.int64), np.zeros(x.size)
    if temperature > 0:
        with np.errstate(invalid="ignore", over="ignore"):
            z = np.where(x == m, 0.0, (x - m) / temperature)
            w = ONE * np.exp(np.where(x == -np.inf, -np.inf, z))
            # z carries three fp32 roundings, exp two units in the last place
            slack = np.where(x == m, 0.0, w * (np.where(np.isfinite(z), -z, 0.0) * 3 + 4) * 2.0 ** -24)
    else:
        w, slack = np.where(x == m, float(ONE), 0.0), np.zeros(x.size)
    return np.rint(w).astype(np.int64), np.where(np.isfinite(slack), slack, 0.0)


def choices(x, temperature, top_k, top_p, min_p, u):
    """{token: [logprobs]} that are right: one unless a decision is within fp32's error of its bound."""
    w, slack = weights(x, temperature)
    if not w.any():
        return {-1: [-math.inf]}
    n = w.size
    k = 1 if temperature <= 0 else (top_k if top_k > 0 else n)
    order = np.lexsort((np.arange(n), -w))[:k]
    order = order[w[order] > 0]
    mass = int(w[order].sum())
    off = float(np.where(slack[order] > 0, slack[order] + 1, 0).sum())  # and the rounding to whole numbers
    before = np.cumsum(w[order]) - w[order]
    found = {}
    target = math.ceil(np.float64(top_p) * mass) if top_p < 1 else mass
    floor_w = math.ceil(np.float64(np.float32(min_p)) * ONE)
    for t in {target, target - 2 * off, target + 2 * off}:
        first = order[(before < t) | (np.arange(order.size) == 0)]
        for sign in (0, -1, 1):
            near = sign * np.where(slack[first] > 0, slack[first] + 1, 0)
            kept = np.sort(first[w[first] + near >= floor_w])
            total = int(w[kept].sum())
            if total == 0:
                found[-1] = [-math.inf]
                continue
            want = math.floor(np.float64(u) * total)
            sums = np.cumsum(w[kept])
            for x0 in (want, want - 2 * off, want + 2 * off):
                i = int(np.searchsorted(sums, min(max(x0, 0), total - 1), side="right"))
                i = min(i, kept.size - 1)
                tok = int(kept[i])
                found.setdefault(tok, []).append(math.log(int(w[tok])) - math.log(total))
    return found


def run(logits, temperature=None, top_k=None, top_p=None, min_p=None, u=None, stream=None):
    rows, vocab = logits.shape
    dev = [None if a is None else torch.tensor(a, dtype=t, device="cuda") for a, t in
           ((temperature, torch.float32), (top_k, torch.int32), (top_p, torch.float32), (min_p, torch.float32), (u, torch.float32))]
    tokens = torch.full((rows + 2,), -7, dtype=torch.int32, device="cuda")
    logp = torch.full((rows + 2,), 7.0, dtype=torch.float32, device="cuda")
    mm.mm_sample(logits, rows, vocab, logits.stride(0), *dev, tokens[1:], logp[1:], stream)
    torch.cuda.synchronize()
    mm.mm_check_device_error()
    t, p = tokens.cpu().numpy(), logp.cpu().numpy()
    assert t[0] == t[-1] == -7 and p[0] == p[-1] == 7.0, "written outside the outputs"
    return t[1:-1], p[1:-1]


def check(logits, temperature, top_k, top_p, min_p, u):
    rows = logits.shape[0]
    tokens, logp = run(logits, temperature, top_k, top_p, min_p, u)
    x = logits.float().cpu().numpy()

    def at(a, r, off):
        return off if a is None else float(np.float32(a[r]))

    several = 0
    for r in range(rows):
        ok = choices(x[r], at(temperature, r, 1.0), int(at(top_k, r, 0)), at(top_p, r, 1.0), at(min_p, r, 0.0), np.float32(u[r]))
        assert int(tokens[r]) in ok, f"row {r}: token {tokens[r]}, not one of {ok}"
        want = min(ok[int(tokens[r])], key=lambda x: 0.0 if x == logp[r] else abs(x - logp[r]))
        # the weight's rounding to a whole number (up to a half of it, for weights of a few units)
        w, slack = weights(x[r], at(temperature, r, 1.0))
        err = 1e-5 + (0 if tokens[r] < 0 else (1.0 + slack[tokens[r]]) / w[tokens[r]])
        assert logp[r] == want or abs(logp[r] - want) <= err * (1 + abs(want)), f"row {r}: logprob {logp[r]}, not {want}"
        several += len(ok) > 1
    assert several <= rows // 2 + 1, "too many rows without a single right token"
    return tokens


def logits_of(seed, rows, vocab, dtype, scale=3.0, offset=0.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((scale * rng.standard_normal((rows, vocab)) + offset).astype(np.float32)).cuda()
    return x.to({"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4099, 20001])
def test_all_filters(vocab, dtype):
    rows = 12
    rng = np.random.default_rng(vocab)
    x = logits_of(vocab, rows, vocab, dtype)
    check(x, rng.uniform(0.4, 1.5, rows), rng.integers(1, 200, rows), rng.uniform(0.5, 1.0, rows), rng.uniform(0, 0.1, rows),
          rng.random(rows))


FILTERS = [dict(), dict(k=40), dict(k=1), dict(k=700), dict(k=100000), dict(p=0.9), dict(p=0.999), dict(p=0.0), dict(m=0.05),
           dict(m=1.0), dict(m=1.5), dict(k=50, p=0.7), dict(k=50, m=0.2), dict(p=0.8, m=0.01), dict(t=0.0), dict(t=-1.0),
           dict(t=1e-3, k=10), dict(t=0.05, p=0.9), dict(t=100.0, k=64, p=0.5), dict(t=100.0, p=0.5)]


@pytest.mark.parametrize("f", FILTERS, ids=[str(sorted(f.items())).replace(" ", "") for f in FILTERS])
def test_each_filter(f):
    rows, vocab = 8, 6001
    rng = np.random.default_rng(5)
    x = logits_of(17, rows, vocab, "f32")
    check(x, [f["t"]] * rows if "t" in f else None, [f["k"]] * rows if "k" in f else None, [f["p"]] * rows if "p" in f else None,
          [f["m"]] * rows if "m" in f else None, rng.random(rows))


@pytest.mark.parametrize("k", [0, 3, 60])
def test_ties_go_to_the_lowest_index(k):
    rows, vocab = 6, 5003
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.integers(-3, 4, (rows, vocab)).astype(np.float32)).half().cuda()
    x[0] = 1.0  # a row of equals
    x[1, 4000:] = float("-inf")
    t = check(x, None, [k] * rows, [0.3] * rows, None, rng.random(rows))
    assert t[0] < vocab
    g = run(x, temperature=[0.0] * rows, u=[0.99] * rows)[0]
    assert g.tolist() == [int(np.argmax(r)) for r in x.float().cpu().numpy()]


def test_masked_infinite_and_nan_logits():
    vocab = 9001
    x = logits_of(9, 10, vocab, "f32")
    low = torch.finfo(torch.float32).min
    x[0] = float("-inf")                                  # nothing left
    x[1] = float("-inf"); x[1, 77] = -5.0                 # one left
    x[2] = low; x[2, [3, 8000]] = torch.tensor([1.0, 1.5], device="cuda")  # masked by the lowest value
    x[3] = low                                            # all of it masked that way: all equal
    x[4, 500] = float("inf")                              # one infinite
    x[5, [9, 700]] = float("inf")
    x[6, ::2] = float("nan")
    x[7] = float("nan")
    x[8, 100:] = float("-inf")
    rng = np.random.default_rng(1)
    for k in (0, 5, 60, 600):
        for p in (1.0, 0.9):
            t = check(x, [0.8] * 10, [k] * 10, [p] * 10, None, rng.random(10))
            assert t[0] == t[7] == -1 and t[1] == 77 and t[4] == 500 and t[2] in (3, 8000) and t[5] in (9, 700) and t[6] % 2 == 1
    # f16's lowest value
    h = x[:3].clamp(min=-60000).half()
    h[2] = -65504.0
    h[2, 5] = 2.0
    assert run(h, top_k=[4] * 3, u=[0.5] * 3)[0][2] == 5


def test_ends_of_u_and_no_logprobs():
    x = logits_of(4, 4, 3001, "bf16")
    check(x, None, [20] * 4, None, None, [0.0, 1 - 2.0 ** -24, 2.0 ** -24, 0.5])
    check(x, None, None, None, None, [0.0, 1 - 2.0 ** -24, 2.0 ** -24, 0.5])
    tokens = torch.empty(4, dtype=torch.int32, device="cuda")
    u = torch.full((4,), 0.25, device="cuda")
    mm.mm_sample(x, 4, 3001, x.stride(0), None, None, None, None, u, tokens, None)
    assert tokens.tolist() == run(x, u=[0.25] * 4)[0].tolist()


def test_strided_rows_streams_and_many_rows():
    # rows inside a wider matrix, at every alignment; NaN between the rows
    wide = torch.full((400, 1037), float("nan"), dtype=torch.float16, device="cuda")
    x = wide[:, 3:1003]
    x.copy_(logits_of(6, 400, 1000, "f16"))
    rng = np.random.default_rng(3)
    a = (rng.uniform(0.5, 1.2, 400), rng.integers(0, 60, 400), rng.uniform(0.6, 1.0, 400), rng.uniform(0, 0.1, 400), rng.random(400))
    t = check(x, *a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert run(x, *a, stream=side)[0].tolist() == t.tolist()


def test_large_vocabulary_and_distribution():
    # 150,001 logits a row; then one row's tokens over evenly spread numbers come out as often as they weigh
    x = logits_of(8, 3, 150001, "f32")
    rng = np.random.default_rng(8)
    check(x, [1.0] * 3, [100, 0, 512], [0.95] * 3, [0.0] * 3, rng.random(3))
    n = 4096
    row = logits_of(12, 1, 512, "f32", scale=1.0)
    t, _ = run(row.expand(n, 512).contiguous(), top_k=[8] * n, u=(np.arange(n) + 0.5) / n)
    w, _ = weights(row.cpu().numpy()[0], 1.0)
    best = np.lexsort((np.arange(512), -w))[:8]
    share = w[best] / w[best].sum()
    count = np.array([(t == b).sum() for b in best]) / n
    assert abs(count - share).max() <= 2 / n and (np.diff(t) >= 0).all()


@pytest.mark.parametrize("rows", [4, 400])  # a row to all of an SM's warps, and four rows to an SM
@pytest.mark.parametrize("what", ["wide", "all equal", "nearly equal", "unaligned", "two values"])
def test_without_the_list(what, rows):
    # top-k off or above 512: sums that pass 32 bits, a bin with more weights than its list, ties over a whole row
    rng = np.random.default_rng(len(what))
    if what == "wide":
        x = logits_of(31, rows, 9001, "f32", scale=6.0)
    elif what == "all equal":
        x = torch.zeros((rows, 140001 if rows < 9 else 5000), dtype=torch.float16, device="cuda")
    elif what == "nearly equal":
        n = 70001 if rows < 9 else 6001
        x = torch.from_numpy(np.stack([-1e-5 * rng.permutation(n) for _ in range(rows)]).astype(np.float32)).cuda()
    elif what == "unaligned":
        x = logits_of(32, rows, 3333, "bf16")[:, 1:3330]
    else:
        x = torch.from_numpy((rng.integers(0, 2, (rows, 4097)) * -0.5).astype(np.float32)).cuda()
    k = [(0, 0, 1000, 5000)[r % 4] for r in range(rows)]
    p = [(0.7, 1.0, 0.9, 1.0)[r % 4] for r in range(rows)]
    q = [(0.0, 0.1, 0.0, 0.2)[(r // 4) % 4] for r in range(rows)]
    check(x, [0.9] * rows, k, p, q, rng.random(rows))


def test_refusals():
    x = logits_of(1, 2, 100, "f32")
    u = torch.zeros(2, device="cuda")
    tokens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(rows=0), dict(vocab=0), dict(stride=99), dict(u=None), dict(tokens=None), dict(vocab=(1 << 24) + 1, stride=1 << 25),
                dict(tokens=x.view(torch.int32)), dict(u=tokens)):
        a = {**dict(logits=x, rows=2, vocab=100, stride=100, temperature=None, top_k=None, top_p=None, min_p=None, u=u, tokens=tokens), **bad}
        with pytest.raises(mm.MMError) as e:
            mm.mm_sample(**a)
        assert e.value.status == mm.MM_ERR_INVALID_ARG, bad
    with pytest.raises(ValueError):
        mm.mm_sample(x.double(), 2, 100, 100, None, None, None, None, u, tokens)
