"""What the Python calls of the cache, its attention and the sampler refuse of a tensor before its address reaches the
library: another type, strides, too few elements, host memory (no GPU needed, nothing is launched)."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import build as mmbuild
from test_abi_cache import P, cache


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mmbuild.build()
    mm.load_library()


def refused(call, why):
    with pytest.raises(mm.MMError) as e:
        call()
    assert e.value.status == mm.MM_ERR_INVALID_ARG and why in str(e.value), e.value


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


# the cache: 3 sequences, 2 kv heads of 64, f16; the calls below are for 5 tokens of 4 heads
ARRAYS = {
    "need": (3, lambda t: mm.mm_cache_reserve(cache(), t, P[6], 0)),
    "missing": (1, lambda t: mm.mm_cache_reserve(cache(), P[5], t, 0)),
    "append q_start": (4, lambda t: mm.mm_cache_append(cache(), 0, P[5], P[6], 128, t, 5, 3, 0)),
    "compact q_start": (4, lambda t: mm.mm_cache_compact(cache(), t, P[6], P[7], 5, 3, 0)),
    "keep": (5, lambda t: mm.mm_cache_compact(cache(), P[5], t, P[7], 5, 3, 0)),
    "kept": (3, lambda t: mm.mm_cache_compact(cache(), P[5], P[6], t, 5, 3, 0)),
    "parents": (2, lambda t: mm.mm_cache_fork(cache(), t, P[6], 2, P[7], 0)),
    "children": (2, lambda t: mm.mm_cache_fork(cache(), P[5], t, 2, P[7], 0)),
    "fork missing": (1, lambda t: mm.mm_cache_fork(cache(), P[5], P[6], 2, t, 0)),
    "list": (2, lambda t: mm.mm_cache_free(cache(), t, 2, 0, 0, 0)),
    "src": (2, lambda t: mm.mm_cache_copy_pages(cache(), t, P[5], 2, 0)),
    "dst": (2, lambda t: mm.mm_cache_copy_pages(cache(), P[5], t, 2, 0)),
    "q_start": (4, lambda t: mm.mm_cache_attention(cache(), 0, P[5], 256, 4, t, 5, 3, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)),
    "tree q_start": (4, lambda t: mm.mm_cache_attention_tree(cache(), 0, P[5], 256, 4, t, 5, 3, P[9], 2, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)),
    "mask": (10, lambda t: mm.mm_cache_attention_tree(cache(), 0, P[5], 256, 4, P[6], 5, 3, t, 2, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)),
}


@pytest.mark.parametrize("name", ARRAYS)
def test_whole_numbers(name):
    n, call = ARRAYS[name]
    refused(lambda: call(i32(n).long()), "int32")
    refused(lambda: call(i32(n).float()), "int32")
    if n > 1:
        refused(lambda: call(i32(2 * n)[::2]), "contiguous")
    refused(lambda: call(i32(n - 1)), "elements")
    refused(lambda: call(i32(n)), "not on the GPU")


HALF = {
    "K": (2, lambda t, row: mm.mm_cache_append(cache(), 0, t, P[6], row, P[7], 5, 3, 0)),
    "V": (2, lambda t, row: mm.mm_cache_append(cache(), 0, P[6], t, row, P[7], 5, 3, 0)),
    "Q": (4, lambda t, row: mm.mm_cache_attention(cache(), 0, t, row, 4, P[6], 5, 3, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)),
    "O": (4, lambda t, row: mm.mm_cache_attention(cache(), 0, P[7], 256, 4, P[6], 5, 3, 0, 0, 0.1, t, row, P[8], 1 << 30, 0)),
    "tree Q": (4, lambda t, row: mm.mm_cache_attention_tree(cache(), 0, t, row, 4, P[6], 5, 3, P[9], 1, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)),
    "tree O": (4, lambda t, row: mm.mm_cache_attention_tree(cache(), 0, P[7], 256, 4, P[6], 5, 3, P[9], 1, 0, 0, 0.1, t, row, P[8], 1 << 30, 0)),
}


@pytest.mark.parametrize("name", HALF)
def test_rows(name):
    heads, call = HALF[name]
    width = heads * 64
    half = lambda *shape: torch.zeros(shape, dtype=torch.float16)
    for other in (torch.float32, torch.bfloat16, torch.int32, torch.uint8):
        refused(lambda: call(half(5, heads, 64).to(other), width), "the cache's type")
    refused(lambda: call(half(heads, 5, 64).transpose(0, 1), 64), "side by side")
    refused(lambda: call(half(5, 64, heads).transpose(1, 2), width), "side by side")
    refused(lambda: call(half(width, 5).T, 1), "side by side")
    refused(lambda: call(half(4, width), width), "ends before")
    refused(lambda: call(half(5, width), width + 8), "ends before")
    # right ones, but for where they lie
    for t, row in ((half(5, heads, 64), width), (half(5, width), width), (half(1, 5, width), width), (half(5 * width), width),
                   (half(5, width + 72)[:, 8:8 + width], width + 72), (half(5, 3 * heads, 64)[:, heads:2 * heads], 3 * width),
                   (half(5, heads, 64).view(torch.int16), width)):
        refused(lambda: call(t, row), "not on the GPU")


def test_bfloat16_cache():
    c, q = cache(dtype=mm.MM_BF16), torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    call = lambda t: mm.mm_cache_attention(c, 0, t, 256, 4, P[6], 5, 3, 0, 0, 0.1, P[7], 256, P[8], 1 << 30, 0)
    refused(lambda: call(q), "not on the GPU")
    refused(lambda: call(q.half()), "the cache's type")


def test_workspace():
    call = lambda t, n: mm.mm_cache_attention(cache(), 0, P[5], 256, 4, P[6], 5, 3, 0, 0, 0.1, P[7], 256, t, n, 0)
    refused(lambda: call(torch.zeros(99, dtype=torch.uint8), 100), "100 contiguous bytes")
    refused(lambda: call(torch.zeros(200, dtype=torch.uint8)[::2], 100), "100 contiguous bytes")
    refused(lambda: call(torch.zeros(25), 100), "not on the GPU")


def test_sampling():
    def call(**a):
        a = {**dict(logits=torch.zeros((2, 100)), rows=2, vocab=100, stride=100, temperature=None, top_k=None, top_p=None,
                    min_p=None, u=P[1], tokens=P[2], logprobs=None, stream=0), **a}
        return lambda: mm.mm_sample(**a)

    on_gpu = "not on the GPU"
    refused(call(), on_gpu)
    refused(call(logits=torch.zeros((100, 2)).T, stride=1), "contiguous")
    refused(call(logits=torch.zeros((1, 100))), "ends before")
    refused(call(logits=torch.zeros((2, 99)), stride=99), "ends before")
    for good, stride in ((torch.zeros(200), 100), (torch.zeros((2, 1, 100)), 100), (torch.zeros((2, 130))[:, 7:107], 130)):
        refused(call(logits=good, stride=stride), on_gpu)
    with pytest.raises(ValueError):
        call(logits=torch.zeros((2, 100), dtype=torch.float64))()


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", "u", "tokens", "logprobs"])
def test_sampling_parameters(name, monkeypatch):
    # (the logits, which are looked at first, pass for the test's sake)
    monkeypatch.setattr(mm, "_reach", lambda *a: None)
    right = torch.int32 if name in ("top_k", "tokens") else torch.float32

    def call(t):
        a = dict(temperature=None, top_k=None, top_p=None, min_p=None, u=P[1], tokens=P[2], logprobs=None)
        return lambda: mm.mm_sample(torch.zeros((2, 100)), 2, 100, 100, **{**a, name: t}, stream=0)

    refused(call(torch.zeros(2, dtype=torch.float64)), str(right))
    refused(call(torch.zeros(2, dtype=torch.int64)), str(right))
    refused(call(torch.zeros(2, dtype=torch.float32 if right == torch.int32 else torch.int32)), str(right))
    refused(call(torch.zeros(4, dtype=right)[::2]), "contiguous")
    refused(call(torch.zeros(1, dtype=right)), "elements")
    refused(call(torch.zeros(2, dtype=right)), "not on the GPU")


def test_cache_on_the_host():
    k = torch.zeros((1, 4, 1, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="on the GPU"):
        mm.mm_cache(k, k.clone(), torch.zeros((2, 3), dtype=torch.int32), i32(2), i32(4))
