"""Offsets whose ranges overlap: reported, nothing written outside Y, and where the ranges together hold more slots than there are,
nothing is written at all (their units of work, up to 512 times as many as the call's sizes allow, would not be numbered by 32 bits)."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import make_weights, make_x, make_y, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


@pytest.mark.parametrize("rows,static", [(100, False), (2000, True)])
@pytest.mark.parametrize("gather", [False, True])
def test_ranges_that_hold_too_many_slots(rows, static, gather):
    experts, slots, cols = 64, 4096, 64
    w, _ = make_weights(1, experts, rows, cols, 32, "f16", static=static)
    torch.cuda.synchronize()
    x, _ = make_x(2, slots, cols, "f16")
    y, buf = make_y(slots, rows, "f32")
    offsets = torch.tensor([0, slots] * (experts // 2) + [0], dtype=torch.int32, device="cuda")
    order = torch.arange(slots, dtype=torch.int32, device="cuda") if gather else None
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), slots, order, 1, offsets, slots, mm.MM_ACT_NONE, y, y.stride(0))
    with pytest.raises(mm.MMError) as e:
        mm.mm_check_device_error()
    assert e.value.status == mm.MM_ERR_INVALID_ARG
    untouched(y, buf)
    assert bool((y == -7).all())


def test_all_ranges_full_to_the_last_slot():
    # the most chunks that ascending offsets give: one slot more than whole chunks for every expert
    experts, rows, cols = 64, 40, 64
    counts = [65] * experts
    w, dense = make_weights(1, experts, rows, cols, 32, "f16")
    n = sum(counts)
    x, xd = make_x(2, n, cols, "f16")
    y, buf = make_y(n, rows, "f32")
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda") * 65
    mm.mm_experts_gemm_packed4(w, x, x.stride(0), n, None, 1, offsets, n, mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    for e in range(experts):
        a = xd[65 * e:65 * e + 65]
        ref, mass = a @ dense[e].T, a.abs() @ dense[e].abs().T
        assert bool(((y[65 * e:65 * e + 65].double().cpu() - ref).abs() <= 1e-5 * mass + 2.0 ** -24 * ref.abs()).all())


def test_the_most_units_in_32_bits():
    """The arithmetic that the limit is for, on the CPU: the largest sizes the call takes and alternating offsets."""
    slots, experts = 1 << 30, 1024
    shortest = -(-slots // 64)
    assert experts // 2 * shortest > 1 << 31                   # chunks of overlapping ranges
    assert 64 * shortest <= 1 << 30                            # a warp's sum, of two experts to a lane
    assert shortest + experts < 1 << 26 and 20 * (1 << 26) < 1 << 31  # the limit, and the sum of clamped warps
