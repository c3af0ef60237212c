"""Sizes, strides and workspaces that the cache calls refuse before any CUDA call (no GPU needed; no pointer passed is ever
dereferenced)."""
import ctypes

import pytest

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import build as mmbuild
from test_abi_cache import P, cache, refused


@pytest.fixture(scope="module")
def lib():
    mmbuild.build()
    return mm.load_library()


BIG = 1 << 38  # the largest stride


@pytest.mark.parametrize("far", [dict(pages=(1 << 31) - 1, page_stride=BIG), dict(pages=1 << 20, page_stride=BIG),
                                 dict(layers=32767, layer_stride=BIG), dict(kv_heads=65535, seqs=1, head_stride=BIG)], ids=str)
def test_a_cache_past_any_memory(lib, far):
    # pages 2^38 elements apart, 2^31 of them: the last one's offset passes 64 bits
    c = cache(**far)
    refused(lib, lib.mm_cache_free(c, P[5], 1, 0, 0, None))
    refused(lib, lib.mm_cache_append(c, 0, P[5], P[6], c.kv_heads * 64, P[7], 5, 3, None))
    refused(lib, lib.mm_cache_attention(c, 0, P[5], c.kv_heads * 64, c.kv_heads, P[6], 5, 3, 0, 0, 0.125, P[7], c.kv_heads * 64, P[8], 1 << 40, None))
    assert "bytes" in lib.mm_last_error().decode()


def test_a_large_cache_is_not(lib):
    # 2^45 elements from end to end: more than there is, but every offset is a number
    n = ctypes.c_int64(-1)
    assert lib.mm_cache_attention_workspace(cache(pages=1 << 20, page_stride=1 << 25), 4, 5, 3, ctypes.byref(n)) == mm.MM_OK and n.value > 0


@pytest.mark.parametrize("heads,tokens,most", [(65534, (1 << 31) - 1, (1 << 31) - 1), (2 << 14, 1 << 20, 1 << 20), (4, (1 << 31) - 1, 1 << 30)])
def test_workspace_of_sizes_that_no_call_takes(lib, heads, tokens, most):
    # the rows of one sequence (new tokens times query heads of a kv head) pass 2^30: attention refuses, and so does this
    c, n = cache(), ctypes.c_int64(-1)
    refused(lib, lib.mm_cache_attention_workspace(c, heads, tokens, most, ctypes.byref(n)))
    assert n.value == -1
    refused(lib, lib.mm_cache_attention(c, 0, P[5], heads * 64, heads, P[6], tokens, most, 0, 0, 0.125, P[7], heads * 64, P[8], 1 << 40, None))


@pytest.mark.parametrize("what", ["k", "v", "the end of v", "table", "lens", "refs", "q_start", "mask", "Q", "O"])
def test_workspace_over_what_the_call_reads_or_keeps(lib, what):
    # the split's partial results would be written over it
    c, last = cache(), 10 * 2048 * 2 * 2 - 16
    at = {"k": P[0], "v": P[1] - 4096 * 2, "the end of v": P[1] + last, "table": P[2], "lens": P[3], "refs": P[4], "q_start": P[6],
          "mask": P[9], "Q": P[5] - 16, "O": P[7] + 256}[what]
    front = (c, 0, P[5], 256, 4, P[6], 5, 3)
    back = (0, 0, 0.125, P[7], 256, at, 1 << 40, None)
    refused(lib, lib.mm_cache_attention_tree(*front, P[9], 1, *back))
    assert "workspace overlaps" in lib.mm_last_error().decode()
    if what != "mask":
        refused(lib, lib.mm_cache_attention(*front, *back))
