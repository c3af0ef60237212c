"""Pairs of CTAs that share an MMA, where one matrix or the experts give units enough: chunks of more than 64 rows of X, unequal
ones, groups of every size, zeros, both types, the activation, static weights, and experts whose rows lie in place.  Sizes are
made from the number of SMs, as the choice is."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import check, make_weights, make_x, make_y, reference, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def rows_for(m, more=0):
    """Rows of W, an even number inside the last tile of 256, that give pairs of CTAs a unit each, and a few more."""
    sms, chunks = torch.cuda.get_device_properties(0).multi_processor_count, -(-m // 256)
    return 256 * (-(-(sms // 2) // chunks) + 2 + more) + 38


def weights(seed, experts, rows, cols, group, dtype, zeros, static):
    w, dense = make_weights(seed, experts, rows, cols, group, dtype, zeros, static=static)
    torch.cuda.synchronize()
    return w, dense.cuda()


CASES = [  # cols, group, dtype, out, zeros, swiglu, static
    (392, 64, "bf16", "bf16", True, False, True), (264, 32, "f16", "f32", True, False, False), (520, 128, "f16", "f16", False, True, True),
    (64, 32, "bf16", "f32", True, True, True), (1000, 128, "bf16", "bf16", True, True, False), (200, 64, "f16", "f16", True, True, False),
    (128, 128, "bf16", "f32", False, False, True), (712, 32, "bf16", "bf16", True, False, True)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("m", [33, 100, 256, 257, 600, 1100])
def test_one_matrix(m, case):
    cols, group, dtype, out, zeros, swiglu, static = case
    rows = rows_for(m, more=m % 5)
    w, dense = weights(m, 1, rows, cols, group, dtype, zeros, static)
    x, xd = make_x(m + 1, m, cols, dtype)
    ref, tol = reference(xd.cuda(), dense[0], swiglu)
    last = None
    for pad in (8, 3, 8):
        y, buf = make_y(m, rows // 2 if swiglu else rows, out, pad=pad)
        mm.mm_gemm_packed4(w, x, x.stride(0), m, mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
        mm.mm_check_device_error()
        untouched(y, buf)
        check(y, ref.cpu(), tol.cpu(), out, f"{m} x {cols} to {rows}")
        assert last is None or torch.equal(last, y)
        last = y.clone()


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("counts", [[300, 257, 0, 1, 900, 64], [70] * 12, [0, 1500, 0, 33]], ids=str)
def test_experts_in_place(counts, case):
    cols, group, dtype, out, zeros, swiglu, static = case
    n, e = sum(counts), len(counts)
    rows = rows_for(n)
    w, dense = weights(n, e, rows, cols, group, dtype, zeros, static)
    slots = n + 5
    x, xd = make_x(n + 1, slots, cols, dtype, bad=range(n, slots))
    y, buf = make_y(slots, rows // 2 if swiglu else rows, out)
    ends = [sum(counts[:i]) for i in range(e + 1)]
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), slots, None, 1, torch.tensor(ends, dtype=torch.int32, device="cuda"), slots,
                               mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    assert bool((y[n:] == -7).all()), "rows behind the last slot were written"
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            ref, tol = reference(xd[a:b].cuda(), dense[i], swiglu)
            check(y[a:b], ref.cpu(), tol.cpu(), out, f"expert {i} of {b - a}")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_experts_gathered(case):
    cols, group, dtype, out, zeros, swiglu, static = case
    counts = [640, 0, 515, 1, 90]
    n, e = sum(counts), len(counts)
    rows = rows_for(n)
    w, dense = weights(3, e, rows, cols, group, dtype, zeros, static)
    x, xd = make_x(4, 700, cols, dtype, bad=(699,))  # no slot names the last row
    order = torch.randint(0, 699 * 2, (n,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    y, buf = make_y(n, rows // 2 if swiglu else rows, out)
    ends = [sum(counts[:i]) for i in range(e + 1)]
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), 700, order.cuda(), 2, torch.tensor(ends, dtype=torch.int32, device="cuda"), n,
                               mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            ref, tol = reference(xd[(order[a:b] // 2).long()].cuda(), dense[i], swiglu)
            check(y[a:b], ref.cpu(), tol.cpu(), out, f"expert {i} of {b - a}")


def test_captured_and_behind_the_call_whose_result_it_takes():
    """Two products in a chain, static weights: the second's X is the first's Y."""
    m, mid = 300, 1024
    first, a = weights(1, 1, mid, 2048, 128, "bf16", True, True)
    rows = rows_for(m)
    second, b = weights(2, 1, rows, mid, 64, "bf16", True, True)
    x, xd = make_x(3, m, 2048, "bf16", pad=0)
    h, y = torch.zeros(m, mid, dtype=torch.bfloat16, device="cuda"), torch.zeros(m, rows, dtype=torch.bfloat16, device="cuda")

    def both():
        mm.mm_gemm_packed4(first, x, 2048, m, mm.MM_ACT_NONE, h, mid)
        mm.mm_gemm_packed4(second, h, mid, m, mm.MM_ACT_NONE, y, rows)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for turn in range(3):
        x.copy_((xd * (turn + 1)).bfloat16())
        h.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        mm.mm_check_device_error()
        check(h, *(t.cpu() for t in reference(x.double(), a[0], False)), "bf16")
        check(y, *(t.cpu() for t in reference(h.double(), b[0], False)), "bf16")
