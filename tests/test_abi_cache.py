"""Argument checks of the cache, attention and sampling calls: each returns its status code before any CUDA call (no GPU
needed), so no pointer passed is ever dereferenced and no kernel is launched, on any machine."""
import ctypes

import pytest

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import build as mmbuild

P = [0x1000000 * (i + 1) for i in range(12)]  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    mmbuild.build()
    return mm.load_library()


def cache(**changes):
    # 2 layers of 10 pages of 2 heads x 16 tokens x 64; 3 sequences of at most 4 pages
    c = mm.Cache(P[0], P[1], P[2], P[3], P[4], 2, 10, 2, 16, 64, 3, 4, 10 * 2048, 2048, 1024, 64, mm.MM_F16)
    for name, value in changes.items():
        setattr(c, name, value)
    return c


BAD_CACHES = [dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(k=P[0] + 8), dict(v=P[1] + 2), dict(table=P[2] + 2),
              dict(layers=0), dict(pages=0), dict(kv_heads=0), dict(seqs=0), dict(max_pages=0), dict(page_size=0), dict(page_size=24),
              dict(page_size=256), dict(head_dim=0), dict(head_dim=68), dict(head_dim=136), dict(dtype=mm.MM_F32), dict(dtype=-1),
              dict(token_stride=60), dict(token_stride=56), dict(max_pages=1 << 27)]


def refused(lib, status):
    assert status == mm.MM_ERR_INVALID_ARG, lib.mm_last_error()
    assert lib.mm_last_error()


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(lib, bad):
    c = cache(**bad)
    refused(lib, lib.mm_cache_append(c, 0, P[5], P[6], 128, P[7], 5, 3, None))
    refused(lib, lib.mm_cache_attention(c, 0, P[5], 256, 4, P[6], 5, 3, 0, 0, 0.125, P[7], 256, P[8], 1 << 30, None))
    refused(lib, lib.mm_cache_free(c, P[5], 1, 0, 0, None))
    n = ctypes.c_int64(-1)
    refused(lib, lib.mm_cache_attention_workspace(c, 4, 5, 3, ctypes.byref(n)))


def test_page_calls(lib):
    c, bare = cache(), cache(refs=None)
    for st in (lib.mm_cache_reserve(None, P[5], P[6], None), lib.mm_cache_reserve(bare, P[5], P[6], None),
               lib.mm_cache_reserve(c, None, P[6], None), lib.mm_cache_reserve(c, P[5], None, None),
               lib.mm_cache_append(c, 2, P[5], P[6], 128, P[7], 5, 3, None), lib.mm_cache_append(c, -1, P[5], P[6], 128, P[7], 5, 3, None),
               lib.mm_cache_append(c, 0, None, P[6], 128, P[7], 5, 3, None), lib.mm_cache_append(c, 0, P[5] + 2, P[6], 128, P[7], 5, 3, None),
               lib.mm_cache_append(c, 0, P[5], P[6], 120, P[7], 5, 3, None), lib.mm_cache_append(c, 0, P[5], P[6], 132, P[7], 5, 3, None),
               lib.mm_cache_append(c, 0, P[5], P[6], 128, None, 5, 3, None), lib.mm_cache_append(c, 0, P[5], P[6], 128, P[7], 0, 3, None),
               lib.mm_cache_append(c, 0, P[5], P[6], 128, P[7], 5, 0, None), lib.mm_cache_append(c, 0, P[5], P[6], 128, P[7], 5, 6, None),
               lib.mm_cache_compact(bare, P[5], None, None, 5, 3, None), lib.mm_cache_compact(c, None, None, None, 5, 3, None),
               lib.mm_cache_compact(c, P[5], P[6], None, 5, 3, None), lib.mm_cache_compact(c, P[5], None, None, 5, 6, None),
               lib.mm_cache_fork(bare, P[5], P[6], 1, P[7], None), lib.mm_cache_fork(c, None, P[6], 1, P[7], None),
               lib.mm_cache_fork(c, P[5], P[6], 0, P[7], None), lib.mm_cache_fork(c, P[5], P[6], 1, None, None),
               lib.mm_cache_free(bare, P[5], 1, 0, 0, None), lib.mm_cache_free(c, P[5], 0, 0, 0, None),
               lib.mm_cache_free(c, P[5], 1, -1, 0, None), lib.mm_cache_free(c, P[5], 1, 4, -1, None),
               lib.mm_cache_copy_pages(c, None, P[5], 1, None), lib.mm_cache_copy_pages(c, P[5], P[6], 0, None)):
        refused(lib, st)


@pytest.mark.parametrize("bad", [
    dict(layer=2), dict(q=None), dict(q=P[5] + 2), dict(q_stride=248), dict(q_stride=257), dict(heads=3), dict(heads=0), dict(starts=None),
    dict(tokens=0), dict(most=0), dict(most=6), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(o=None), dict(o=P[5] + 512), dict(o=P[7] + 8), dict(o_stride=248), dict(ws=None, bytes=0), dict(ws=P[8] + 4),
], ids=str)
def test_attention(lib, bad):
    a = {**dict(layer=0, q=P[5], q_stride=256, heads=4, starts=P[6], tokens=5, most=3, window=0, sinks=0, scale=0.125, o=P[7],
                o_stride=256, ws=P[8], bytes=1 << 40), **bad}
    front = (cache(), a["layer"], a["q"], a["q_stride"], a["heads"], a["starts"], a["tokens"], a["most"])
    back = (a["window"], a["sinks"], a["scale"], a["o"], a["o_stride"], a["ws"], a["bytes"], None)
    if "ws" not in bad:  # the workspace's size goes by the device's SMs
        refused(lib, lib.mm_cache_attention(*front, *back))
        refused(lib, lib.mm_cache_attention_tree(*front, P[9], 1, *back))
    refused(lib, lib.mm_cache_attention_tree(*front, None, 1, *back))
    refused(lib, lib.mm_cache_attention_tree(*front, P[9], 0, *back))


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=P[0] + 1), dict(dtype=3), dict(dtype=-1), dict(rows=0), dict(vocab=0), dict(vocab=(1 << 24) + 1),
    dict(stride=999), dict(u=None), dict(u=P[1] + 2), dict(tokens=None), dict(tokens=P[0] + 4), dict(logprobs=P[0]), dict(top_k=P[4] + 1),
], ids=str)
def test_sample(lib, bad):
    a = {**dict(logits=P[0], dtype=mm.MM_F32, rows=2, vocab=1000, stride=1000, temperature=None, top_k=None, top_p=None, min_p=None,
                u=P[1], tokens=P[2], logprobs=P[3]), **bad}
    refused(lib, lib.mm_sample(*a.values(), None))
