"""GPU parity of attention over a paged cache (mm_cache_attention, mm_cache_attention_tree) against the
definition in fp64: ragged batches, grouped heads, windows and sinks, draft trees, head dimensions, page
sizes, strides; rows that see nothing; NaN and infinities where no row, or not every row, looks.

The tolerance of every element is derived in cache_util.tolerance from the roundings the call documents.
"""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import (DT, attention64, check_attention, make_cache, pack_bits, run_attention, starts, tree_bits,
                        visible)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def queries(seed, tokens, heads, dim, dtype, scale=1.5):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((scale * rng.standard_normal((tokens, heads, dim))).astype(np.float32)).to(DT[dtype]).cuda()


# (name, lens, new, heads, kv_heads, dim, page, window, sinks)
CAUSAL = [
    ("one token on nothing", [0], [1], 2, 2, 64, 16, 0, 0),
    ("one token", [37], [1], 4, 2, 64, 16, 0, 0),
    ("page boundaries", [15, 16, 17, 127, 128, 129], [1] * 6, 2, 1, 64, 16, 0, 0),
    ("empty sequences among others", [40, 0, 9, 300], [1, 0, 0, 1], 6, 2, 128, 32, 0, 0),
    ("split keys", [5000, 3, 2049], [1, 1, 1], 8, 1, 128, 64, 0, 0),
    ("16 heads of one", [700], [1], 16, 1, 64, 128, 0, 0),
    ("odd dim", [333, 20], [1, 1], 6, 2, 80, 16, 0, 0),
    ("dim 8", [70], [1], 1, 1, 8, 16, 0, 0),
    ("dim 120", [210], [1], 3, 1, 120, 32, 0, 0),
    ("window", [900, 10, 64, 65], [1, 1, 1, 1], 4, 2, 64, 16, 64, 0),
    ("window and sinks", [900, 10, 64, 69], [1, 1, 1, 1], 4, 2, 128, 16, 64, 5),
    ("window of one", [33], [1], 2, 2, 64, 16, 1, 0),
    ("sinks over the whole", [50], [1], 2, 2, 64, 16, 7, 100),
    ("few new tokens", [100, 31, 0], [4, 1, 3], 4, 1, 64, 16, 0, 0),
    ("few new tokens, window", [100, 31, 0], [4, 2, 3], 4, 1, 128, 32, 6, 2),
    ("17 rows", [250], [17], 1, 1, 64, 16, 0, 0),
    ("chunks", [0, 130, 77], [130, 1, 64], 4, 2, 64, 16, 0, 0),
    ("chunks, group 3", [0, 333], [150, 129], 6, 2, 128, 64, 0, 0),
    ("chunks, group 7, odd dim", [65, 0], [40, 37], 7, 1, 96, 32, 0, 0),
    ("chunks, window", [0, 500, 260], [200, 140, 1], 2, 1, 64, 16, 90, 0),
    ("chunks, window and sinks", [10, 700, 260], [200, 140, 0], 4, 2, 128, 128, 100, 9),
    ("chunk of a long one", [2900], [70], 8, 2, 128, 64, 0, 0),
    ("512 rows on 128 keys", [0], [128], 4, 1, 64, 128, 0, 0),
    ("24 heads of one", [300, 5], [1, 1], 24, 1, 64, 16, 0, 0),
    ("130 heads of one", [300], [2], 130, 1, 64, 16, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", CAUSAL, ids=[c[0].replace(" ", "_").replace(",", "") for c in CAUSAL])
def test_parity(case, dtype):
    _, lens, new, heads, kv_heads, dim, page, window, sinks = case
    c, dk, dv = make_cache(11 + dim, lens, new, kv_heads, dim, page, dtype)
    q = queries(5, sum(new), heads, dim, dtype)
    worst, _ = check_attention(c, dk, dv, 0, q, new, lens, window, sinks, dim ** -0.5, dtype)
    print(f"worst error {worst:.3f} of the tolerance")


# (lens, new, heads, kv_heads, dim, page, window, sinks)
TREES = [
    ([0], [1], 1, 1, 64, 16, 0, 0),
    ([100, 17, 0], [7, 1, 5], 2, 2, 64, 16, 0, 0),
    ([200, 31], [16, 12], 1, 1, 128, 16, 0, 0),
    ([333, 64, 5], [33, 20, 0], 4, 1, 64, 16, 0, 0),
    ([150], [64], 8, 2, 128, 64, 0, 0),
    ([60, 700], [100, 70], 3, 1, 80, 32, 0, 0),
    ([500, 40], [9, 9], 2, 2, 64, 16, 50, 4),
    ([500, 40], [40, 33], 4, 1, 128, 16, 50, 4),
    ([5000], [31], 4, 1, 128, 64, 0, 0),
    ([300], [5], 2, 2, 64, 16, 1, 0),
    ([300], [200], 1, 1, 64, 16, 20, 3),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", TREES, ids=[f"{t[1]}on{t[0]}" for t in TREES])
def test_tree_parity(case, dtype):
    lens, new, heads, kv_heads, dim, page, window, sinks = case
    rng = np.random.default_rng(3)
    c, dk, dv = make_cache(23, lens, new, kv_heads, dim, page, dtype)
    q = queries(6, sum(new), heads, dim, dtype)
    bits = [tree_bits(rng, n) for n in new]
    words = -(-max(new) // 32) + 1  # a wider mask than needed, its unused bits set
    rows = np.ones((sum(new), words * 32), dtype=bool)
    st = starts(new)
    for s, n in enumerate(new):
        rows[st[s]:st[s + 1], :n] = bits[s]
    worst, _ = check_attention(c, dk, dv, 0, q, new, lens, window, sinks, dim ** -0.5, dtype, bits=bits,
                               mask=pack_bits(rows, words).cuda())
    print(f"worst error {worst:.3f} of the tolerance")


def test_one_workspace_for_calls_of_any_size():
    # one after the other in both kernels, with more and with fewer units, heads and columns: each as with its own workspace
    dtype = "f16"
    calls = []
    for seed, (lens, new, heads, kv_heads, dim) in enumerate([([3000, 900], [1, 1], 8, 2, 128), ([5000], [1], 1, 1, 64),
                                                              ([40, 1700, 300], [600, 300, 90], 8, 4, 64), ([700] * 40, [1] * 40, 16, 8, 64),
                                                              ([2500], [40], 4, 1, 128), ([100] * 30, [300] * 30, 8, 8, 64)]):
        c, _, _ = make_cache(seed, lens, new, kv_heads, dim, 64, dtype)
        q = queries(seed, sum(new), heads, dim, dtype)
        calls.append((c, q, new, run_attention(c, 0, q, new, 0, 0, 0.1),
                      mm.mm_cache_attention_workspace(c, heads, sum(new), max(new))))
    ws = torch.zeros(max(need for *_, need in calls), dtype=torch.uint8, device="cuda")
    for i in (0, 5, 1, 2, 3, 4, 0, 2, 5, 3, 1, 0, 4, 2):
        c, q, new, alone, _ = calls[i]
        assert torch.equal(alone.view(torch.int16), run_attention(c, 0, q, new, 0, 0, 0.1, ws=ws).view(torch.int16)), i


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new", [[1, 3, 2], [40, 90, 33]])
@pytest.mark.parametrize("lens,window,sinks", [([300, 45, 16], 24, 3), ([319, 64, 40], 16, 0), ([301, 48, 39], 40, 17)])
def test_pages_released_under_a_window(lens, window, sinks, new, tree):
    # a block of keys reaches into pages that mm_cache_free has taken: no error, and their contents do not show
    dtype, rng = "f16", np.random.default_rng(17)
    c, dk, dv = make_cache(31, lens, new, 2, 64, 16, dtype)
    k, v, table, _, refs = c.tensors
    before = int((table >= 0).sum())
    seqs = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    mm.mm_cache_free(c, seqs, len(lens), window, sinks)
    assert int((table >= 0).sum()) < before
    k[:, refs == 0] = float("nan")
    v[:, refs == 0] = float("nan")
    q = queries(4, sum(new), 4, 64, dtype)
    bits = [tree_bits(rng, n) for n in new] if tree else None
    mask = None
    if tree:
        words = -(-max(new) // 32)
        mask = pack_bits(np.concatenate([np.pad(b, ((0, 0), (0, words * 32 - b.shape[1]))) for b in bits]), words).cuda()
    check_attention(c, dk, dv, 0, q, new, lens, window, sinks, 0.125, dtype, bits=bits, mask=mask)


@pytest.mark.parametrize("layout", ["tokens", "padded", "both"])
@pytest.mark.parametrize("new", [[1, 1], [50, 90]])
def test_layouts_layers_and_strides(layout, new):
    # any order of heads and tokens, padded rows, K and V in one allocation; a layer other than the first;
    # Q a slice of a wider fused row; O with a padded row
    lens, dtype = [300, 45], "f16"
    c, dk, dv = make_cache(9, lens, new, 2, 64, 16, dtype, layers=3, layout=layout)
    wide = queries(8, sum(new), 12, 64, dtype)
    q = wide[:, 4:8]
    for layer in (0, 2):
        check_attention(c, dk, dv, layer, q, new, lens, 0, 0, 0.125, dtype, pad=8)


@pytest.mark.parametrize("heads,new,dim", [(4, [1, 1, 1], 64), (4, [3, 2, 1], 128), (4, [60, 40, 1], 64), (8, [130, 5, 40], 128)])
def test_infinities_and_nan_in_masked_places(heads, new, dim):
    # keys and values that no row sees, and drafted or windowed ones that only some rows see
    dtype, lens, window, sinks = "f16", [400, 77, 30], 48, 3
    c, dk, dv = make_cache(31, lens, new, 2, dim, 16, dtype)
    q = queries(7, sum(new), heads, dim, dtype)
    clean = run_attention(c, 0, q, new, window, sinks, 0.1)
    k, v = c.tensors[0], c.tensors[1]
    table = c.tensors[2].cpu().numpy()
    rng = np.random.default_rng(1)
    values = [float("nan"), float("inf"), float("-inf")]
    for s, n in enumerate(lens):
        ok = visible(n, new[s], window, sinks)
        for j in np.flatnonzero(~ok.any(0)):
            for t, x in ((k, values[j % 3]), (v, values[(j + 1) % 3])):
                t[0, int(table[s, j // 16]), :, int(j % 16)] = x
    again = run_attention(c, 0, q, new, window, sinks, 0.1)
    assert torch.equal(clean.view(torch.int16), again.view(torch.int16))
    # now a value that only some rows see: those get infinity or NaN in that column, the others nothing
    for s, n in enumerate(lens):
        ok = visible(n, new[s], window, sinks)
        some = np.flatnonzero(ok.any(0) & ~ok.all(0))
        if some.size == 0:
            continue
        j = int(some[rng.integers(some.size)])
        v[0, int(table[s, j // 16]), 1, j % 16, 5] = float("inf")
        got = run_attention(c, 0, q, new, window, sinks, 0.1)
        st = starts(new)
        for i in range(new[s]):
            row, was = got[st[s] + i], clean[st[s] + i]
            group = heads // 2
            if ok[i, j]:
                assert bool((~torch.isfinite(row[group:, 5])).all())
                row, was = row.clone(), was.clone()
                row[group:, 5] = was[group:, 5] = 0
            assert bool(torch.isfinite(row).all())
            assert bool(((row - was).abs().float() <= 4e-3 * (1 + was.abs().float())).all())
        v[0, int(table[s, j // 16]), 1, j % 16, 5] = 0.25
        clean = run_attention(c, 0, q, new, window, sinks, 0.1)


@pytest.mark.parametrize("n,heads", [(6, 2), (40, 4)])
def test_tree_rows_that_see_nothing(n, heads):
    # no cached token and no bit: the row is 0; NaN in a draft that only others see leaves it 0
    dtype = "bf16"
    c, dk, dv = make_cache(2, [0, 50], [n, n], 1, 64, 16, dtype)
    q = queries(3, 2 * n, heads, 64, dtype)
    rng = np.random.default_rng(0)
    bits = [tree_bits(rng, n), tree_bits(rng, n)]
    bits[0][2] = False
    bits[1][3] = False
    for b in bits:
        b[:, 4] = False
        b[4, 4] = True  # draft 4 is seen by itself alone
    rows = np.concatenate(bits)
    mask = pack_bits(rows, -(-n // 32)).cuda()
    worst, out = check_attention(c, dk, dv, 0, q, [n, n], [0, 50], 0, 0, 0.125, dtype, bits=bits, mask=mask)
    assert bool((out[2] == 0).all())
    v = c.tensors[1]
    page = int(c.tensors[2][0, 0])
    v[0, page, 0, 4] = float("nan")
    again = run_attention(c, 0, q, [n, n], 0, 0, 0.125, mask=mask)
    assert bool(torch.isnan(again[4]).all())
    again[4] = out[4]  # every other row is as the definition has it
    check_attention(c, dk, dv, 0, q, [n, n], [0, 50], 0, 0, 0.125, dtype, bits=bits, out=again)


@pytest.mark.parametrize("lens,new", [([900, 33], [1, 1]), ([700, 0], [100, 80])])
def test_sharp_scores_and_large_values(lens, new):
    # queries that make each row's softmax sharp: the running reference moves from block to block
    dtype = "f16"
    c, dk, dv = make_cache(77, lens, new, 2, 64, 16, dtype)
    q = queries(12, sum(new), 4, 64, dtype, scale=12.0)
    check_attention(c, dk, dv, 0, q, new, lens, 0, 0, 0.25, dtype)


@pytest.mark.parametrize("lens,new,heads", [([9000, 100], [1, 1], 4), ([3000], [40], 8), ([400, 0], [200, 300], 4)])
def test_runs_are_bit_identical_and_the_workspace_is_reusable(lens, new, heads):
    dtype = "bf16"
    c, dk, dv = make_cache(5, lens, new, 2, 128, 64, dtype)
    q = queries(4, sum(new), heads, 128, dtype)
    ws = torch.zeros(max(16, mm.mm_cache_attention_workspace(c, heads, sum(new), max(new))), dtype=torch.uint8, device="cuda")
    a = run_attention(c, 0, q, new, 0, 0, 0.09, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        b = run_attention(c, 0, q, new, 0, 0, 0.09, ws=ws, stream=side if i % 2 else None)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_far_offsets():
    # strides whose byte offsets pass 2^32: pages 96 MB apart in one allocation of 6 GB
    dtype, page, dim, kv = "f16", 16, 64, 2
    stride = 48 * 1024 * 1024
    pages = 63
    pool = torch.empty(pages * stride, dtype=torch.float16, device="cuda")
    k = pool.as_strided((1, pages, kv, page, dim), (stride * pages, stride, page * dim, dim, 1))
    v = pool[4096:].as_strided((1, pages, kv, page, dim), (stride * pages, stride, page * dim, dim, 1))
    rng = np.random.default_rng(8)
    for new in (1, 60):
        lens = 15 * 16 - 3
        n = lens + new
        held = -(-n // page)
        data = [torch.from_numpy(rng.standard_normal((kv, held * page, dim)).astype(np.float32)).half() for _ in range(2)]
        order = np.array([pages - 1] + list(range(30, 30 + held - 1)), dtype=np.int32)
        for t, d in ((k, data[0]), (v, data[1])):
            for i, p in enumerate(order.tolist()):
                t[0, p] = d[:, i * page:(i + 1) * page].cuda()
        c = mm.mm_cache(k, v, torch.from_numpy(order[None, :].copy()).cuda(), torch.tensor([lens], dtype=torch.int32, device="cuda"))
        q = queries(1, new, 4, dim, dtype)
        dk = [data[0][None, :, :n].double().numpy()]
        dv = [data[1][None, :, :n].double().numpy()]
        check_attention(c, dk, dv, 0, q, [new], [lens], 0, 0, 0.125, dtype)


@pytest.mark.parametrize("new,heads", [([1, 1], 2), ([40, 40], 4)])
def test_out_of_range_metadata_is_reported(new, heads):
    # pages and lengths that the device finds out of range: skipped, and reported once
    dtype = "f16"
    c, dk, dv = make_cache(3, [100, 40], new, 2, 64, 16, dtype)
    q = queries(3, sum(new), heads, 64, dtype)
    good = run_attention(c, 0, q, new, 0, 0, 0.125)
    table, lens = c.tensors[2], c.tensors[3]
    saved = table.clone()
    table[0, 2] = 1 << 20
    with pytest.raises(mm.MMError) as e:
        run_attention(c, 0, q, new, 0, 0, 0.125)
    assert e.value.status == mm.MM_ERR_INVALID_ARG and "out of range" in str(e.value)
    table.copy_(saved)
    lens[1] = 1 << 30
    with pytest.raises(mm.MMError) as e:
        run_attention(c, 0, q, new, 0, 0, 0.125)
    assert e.value.status == mm.MM_ERR_INVALID_ARG
    lens[1] = 40
    assert torch.equal(good, run_attention(c, 0, q, new, 0, 0, 0.125))


def test_refusals():
    c, _, _ = make_cache(3, [20], [2], 2, 64, 16, "f16")
    q = queries(1, 2, 4, 64, "f16")
    o = torch.empty_like(q)
    qs = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    ok = dict(layer=0, Q=q, q_stride=256, heads=4, q_start=qs, tokens=2, max_q=2, window=0, sinks=0, scale=0.125, O=o,
              o_stride=256, workspace=ws, workspace_bytes=ws.numel())
    mm.mm_cache_attention(c, **ok)
    bad = [dict(layer=1), dict(layer=-1), dict(Q=None), dict(O=None), dict(q_stride=255), dict(q_stride=248), dict(heads=3),
           dict(heads=0), dict(tokens=0), dict(max_q=0), dict(max_q=3), dict(window=-1), dict(sinks=-1),
           dict(scale=float("inf")), dict(O=q), dict(o_stride=128), dict(q_start=None), dict(Q=q.data_ptr() + 2)]
    for b in bad:
        with pytest.raises(mm.MMError) as e:
            mm.mm_cache_attention(c, **{**ok, **b})
        assert e.value.status == mm.MM_ERR_INVALID_ARG, b
    mask = torch.ones((2, 1), dtype=torch.int32, device="cuda")
    for b in (dict(mask=None, mask_words=1), dict(mask=mask, mask_words=0)):
        with pytest.raises(mm.MMError):
            mm.mm_cache_attention_tree(c, **{**ok, **b})
    # a workspace that is too small for the split
    big, _, _ = make_cache(3, [4000], [1], 1, 64, 16, "f16")
    q1 = queries(1, 1, 1, 64, "f16")
    need = mm.mm_cache_attention_workspace(big, 1, 1, 1)
    assert need > 0
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for b in (dict(workspace=None), dict(workspace=ws, workspace_bytes=need - 1)):
        with pytest.raises(mm.MMError) as e:
            mm.mm_cache_attention(big, **{**ok, **dict(Q=q1, q_stride=64, heads=1, q_start=one, tokens=1, max_q=1,
                                                       O=torch.empty_like(q1), o_stride=64), **b})
        assert e.value.status == mm.MM_ERR_INVALID_ARG and "workspace" in str(e.value)
    mm.mm_check_device_error()
