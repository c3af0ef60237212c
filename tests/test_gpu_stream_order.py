"""Stream order around calls that start early.  An independent packed GEMV does not wait for the kernel before it, and the
cache and sampling calls wait for the kernel before them alone: what is queued behind an independent call must still find
the results of everything in front of it, and an independent call behind a cache call must not run into what is in front
of that one.  (Each sequence is repeated with other data, so that a result from the time before shows.)
"""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import make_cache, run_attention, starts
from dense_packed_bit_gb300 import synth

pytestmark = pytest.mark.gpu

ROWS, COLS, BATCH, PER_CTA = 1270, 4096, 256, 64  # 2,560 tiles of 127 rows, 64 to a CTA: 40 CTAs, the other SMs stay free

CODEBOOK = np.array([-1.5, -0.5, 0.5, 1.5], dtype=np.float32)  # evenly spaced, as most decodes want it


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


class Long:
    """y[BATCH * ROWS] from 40 CTAs that take 330 MB of codes between them: much longer than what follows it."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(3)
        self.codes = torch.randint(0, 256, (BATCH, ROWS * COLS // 4), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        self.scales = torch.from_numpy(synth.uniform_f16_bits(4, (BATCH * ROWS,), 0.01, 0.02)).cuda()
        self.y = torch.empty(BATCH * ROWS, dtype=torch.float32, device="cuda")
    def __call__(self, x):
        mm.mm_gemv_packed2_strided_batched_ex(self.codes, ROWS * COLS // 4, self.scales, ROWS, x, 0, self.y, ROWS, BATCH, ROWS, COLS,
                                              CODEBOOK, dequant=mm.MM_DEQ_MXF4, rows_per_lane=PER_CTA, pdl=1)


def vectors(n, cols):
    return [torch.from_numpy(synth.normal_f32(20 + i, (cols,), 1.0)).cuda().half() for i in range(n)]


class Short:
    """127 rows of 512 columns, independent, by one of the decodes: a few microseconds."""

    def __init__(self, dequant, batched=False, **opts):
        self.codes = torch.from_numpy(synth.ternary_field_bytes(9, 127 * 128)).cuda()
        self.scales = torch.from_numpy(synth.uniform_f16_bits(10, (127,), 0.5, 1.0)).cuda()
        self.y, self.batched = torch.zeros(127, dtype=torch.float32, device="cuda"), batched
        self.opts = dict(dequant=dequant, pdl=1, independent=1, **opts)

    def __call__(self, x, y=None):
        y = self.y if y is None else y
        if self.batched:
            mm.mm_gemv_packed2_strided_batched_ex(self.codes, 127 * 128, self.scales, 127, x, 0, y, 127, 1, 127, 512,
                                                  CODEBOOK, **self.opts)
        else:
            mm.mm_gemv_packed2_ex(self.codes, self.scales, x, y, 127, 512, CODEBOOK, **self.opts)


class Short4:
    """The same by the 4-bit decode."""

    def __init__(self):
        self.codes = torch.from_numpy(synth.ternary_field_bytes(9, 127 * 256)).cuda()
        self.scales = torch.from_numpy(synth.uniform_f16_bits(10, (127,), 0.5, 1.0)).cuda()
        self.y = torch.zeros(127, dtype=torch.float32, device="cuda")
        self.opts = dict(pdl=1, independent=1, staging=1)

    def __call__(self, x):
        mm.mm_gemv_packed4_ex(self.codes, self.scales, x, self.y, 127, 512, np.linspace(-1, 1, 16).tolist(), **self.opts)


SHORT = {
    "registers": lambda: Short(mm.MM_DEQ_AFFINE, staging=0),
    "select": lambda: Short(mm.MM_DEQ_SELECT, staging=0),
    "staged": lambda: Short(mm.MM_DEQ_AFFINE, staging=1),
    "mma": lambda: Short(mm.MM_DEQ_MMA, staging=0),
    "mma, one warp a row": lambda: Short(mm.MM_DEQ_MMA, staging=0, split=1, warps=1),
    "mma staged": lambda: Short(mm.MM_DEQ_MMA, staging=1),
    "fp8": lambda: Short(mm.MM_DEQ_FP8),
    "tc": lambda: Short(mm.MM_DEQ_TC),
    "fp4": lambda: Short(mm.MM_DEQ_MXF4),
    "batched": lambda: Short(mm.MM_DEQ_MXF4, batched=True),
    "4 bits": Short4,
}


@pytest.fixture(scope="module")
def long():
    return Long()


def first_largest(y):
    tokens = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    u = torch.zeros(1, device="cuda")
    zero = torch.zeros(1, device="cuda")
    return tokens, lambda: mm.mm_sample(y, 1, y.numel(), y.numel(), zero, None, None, None, u, tokens)


@pytest.mark.parametrize("short", SHORT, ids=[s.replace(" ", "_").replace(",", "") for s in SHORT])
def test_sampling_behind_an_independent_gemv(long, short):
    between = SHORT[short]()
    xs, small = vectors(6, COLS), vectors(1, 512)[0]
    tokens, sample = first_largest(long.y)
    want = []
    for x in xs:
        long(x)
        torch.cuda.synchronize()
        want.append(int(long.y.argmax()))
    assert len(set(want)) > 1
    for x, w in zip(xs, want):
        long(x)
        between(small)
        sample()
        assert tokens.item() == w
    mm.mm_check_device_error()


def test_a_row_of_independent_calls(long):
    # the last of them starts beside the long call too
    between = [SHORT[s]() for s in ("staged", "registers", "fp8", "4 bits")]
    xs, small = vectors(4, COLS), vectors(1, 512)[0]
    tokens, sample = first_largest(long.y)
    for x in xs:
        long(x)
        for b in between * 2:
            b(small)
        sample()
        got = tokens.item()
        assert got == int(long.y.argmax())
    mm.mm_check_device_error()


def test_an_independent_call_behind_a_cache_call(long):
    # the long call and the batched one write the same place; the cache call between them makes their order the stream's
    k, v = (torch.zeros((1, 4, 1, 16, 8), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.full((1, 2), -1, dtype=torch.int32, device="cuda")
    one = lambda n: torch.full((1,), n, dtype=torch.int32, device="cuda")
    cache = mm.mm_cache(k, v, table, one(0), torch.zeros(4, dtype=torch.int32, device="cuda"))
    need, missing = one(20), one(0)
    batched, xs, small = SHORT["batched"](), vectors(3, COLS), vectors(1, 512)[0]
    batched(small)
    torch.cuda.synchronize()
    want = batched.y.clone()
    for x in xs:
        for at in (0, (BATCH - 1) * ROWS):
            long(x)
            mm.mm_cache_reserve(cache, need, missing)
            batched(small, long.y[at:at + 127])
            torch.cuda.synchronize()
            assert torch.equal(long.y[at:at + 127], want)
    mm.mm_check_device_error()


@pytest.mark.parametrize("lens,new,heads", [([900, 40], [1, 1], 4), ([300, 0], [20, 90], 4)])
def test_attention_and_sampling_on_another_stream(lens, new, heads):
    # the outputs are made on this stream, and ordered before the call on the other
    c, _, _ = make_cache(5, lens, new, 2, 64, 16, "f16")
    rng = np.random.default_rng(4)
    q = torch.from_numpy(rng.standard_normal((sum(new), heads, 64)).astype(np.float32)).half().cuda()
    want = run_attention(c, 0, q, new, 0, 0, 0.125)
    qs = torch.from_numpy(starts(new)).cuda()
    need = mm.mm_cache_attention_workspace(c, heads, sum(new), max(new))
    logits = torch.from_numpy(rng.standard_normal((3, 5003)).astype(np.float32)).cuda()
    u = torch.full((3,), 0.3, device="cuda")
    k = torch.full((3,), 50, dtype=torch.int32, device="cuda")
    token = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    mm.mm_sample(logits, 3, 5003, 5003, None, k, None, None, u, token)
    side = torch.cuda.Stream()
    for _ in range(5):
        out = torch.full_like(q, 7.0)
        got = torch.full_like(token, -7)
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        mm.mm_cache_attention(c, 0, q, q.stride(0), heads, qs, sum(new), max(new), 0, 0, 0.125, out, out.stride(0), ws, ws.numel(), side)
        mm.mm_sample(logits, 3, 5003, 5003, None, k, None, None, u, got, None, side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(got, token)
    mm.mm_check_device_error()
