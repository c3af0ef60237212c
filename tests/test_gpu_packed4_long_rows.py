"""4-bit products of rows of many groups: the error stays within the bound at any length, also where every addition of a group's
sum is off to the same side; and infinities stay infinities in the compensated totals."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import check, make_weights, make_x, make_y, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def bound(cols, group):
    """1e-5 for 128 groups, and 2^-24 (an fp32 addition) for each further one of 1024."""
    return 1e-5 + 2.0 ** -24 * max(0, min(-(-cols // group), 1024) - 128)


def same_sign(kind, experts, rows, cols, group, n, seed):
    """Weights and X of positive terms: equal ones; random ones; a first group of 2^15 and the others just below half a place
    of it, which plain fp32 sums lose."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = torch.full((experts, rows, cols // 2), 0x11, dtype=torch.uint8, device="cuda")
    x = torch.zeros(n, cols, dtype=torch.float16, device="cuda")
    if kind == "equal":
        x += 1 + 2.0 ** -10
    elif kind == "random":
        byte |= torch.randint(0, 256, byte.shape, generator=g, dtype=torch.uint8, device="cuda")
        x += torch.rand(n, cols, generator=g, device="cuda").half() + 0.125
    else:
        x[:, :group] = 2.0 ** 15 / group
        x[:, group::group] = 0.99 * 2.0 ** -10
    scales = torch.ones(experts, rows, cols // group, dtype=torch.float16, device="cuda")
    if kind != "lost":
        scales *= (0.5 + torch.rand(experts, rows, 1, generator=g, device="cuda")).half()
    return mm.mm_packed4(byte, scales, torch.zeros_like(scales, dtype=torch.uint8), cols, group), byte, scales, x


def exact(byte, scales, group, x):
    """X W^T of one matrix in fp64 on the GPU, a stretch of the columns at a time."""
    y, step = 0, 1 << 19
    for k in range(0, x.shape[1], step):
        b = byte[:, k // 2:(k + step) // 2]
        w = torch.stack([b & 15, b >> 4], -1).flatten(-2).double() * scales[:, k // group:(k + step) // group].double().repeat_interleave(group, -1)
        y = y + x[:, k:k + step].double() @ w.T
    return y


@pytest.mark.parametrize("kind", ["equal", "random", "lost"])
@pytest.mark.parametrize("m,cols,group", [(1, 1 << 22, 32), (12, 1 << 22, 32), (64, 1 << 20, 32), (300, 1 << 20, 32), (64, 1 << 21, 128), (20, 1 << 16, 32)])
def test_same_signs(m, cols, group, kind):
    rows = 24
    w, byte, scales, x = same_sign(kind, 1, rows, cols, group, m, m)
    y = torch.empty(m, rows, device="cuda")
    mm.mm_gemm_packed4(w, x, cols, m, mm.MM_ACT_NONE, y, rows)
    mm.mm_check_device_error()
    ref = exact(byte[0], scales[0], group, x)
    assert bool(((y.double() - ref).abs() <= (bound(cols, group) + 2.0 ** -24) * ref).all()), ((y.double() - ref).abs() / ref).max()


@pytest.mark.parametrize("kind", ["equal", "lost"])
@pytest.mark.parametrize("counts", [[3, 0, 2], [41, 0, 70]])
def test_same_signs_of_experts(counts, kind):
    rows, cols, group, n = 24, 1 << 20, 32, sum(counts)
    w, byte, scales, x = same_sign(kind, len(counts), rows, cols, group, n, 1)
    ends = [sum(counts[:i]) for i in range(len(counts) + 1)]
    y = torch.empty(n, rows, device="cuda")
    mm.mm_experts_gemm_packed4(w, x, cols, n, None, 1, torch.tensor(ends, dtype=torch.int32, device="cuda"), n, mm.MM_ACT_NONE, y, rows)
    mm.mm_check_device_error()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            ref = exact(byte[e], scales[e], group, x[a:b])
            assert bool(((y[a:b].double() - ref).abs() <= (bound(cols, group) + 2.0 ** -24) * ref).all()), ((y[a:b].double() - ref).abs() / ref).max()


@pytest.mark.parametrize("m", [5, 40, 130])
@pytest.mark.parametrize("swiglu", [False, True])
def test_odd_long_rows(m, swiglu):
    rows, cols, group = 38, (1 << 19) + 72, 32
    w, dense = make_weights(m, 1, rows, cols, group, "bf16")
    x, xd = make_x(m + 1, m, cols, "bf16")
    y, buf = make_y(m, rows // 2 if swiglu else rows, "f32")
    mm.mm_gemm_packed4(w, x, x.stride(0), m, mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    d = dense[0]
    z, t = xd @ d.T, bound(cols, group) * (xd.abs() @ d.abs().T)
    if swiglu:  # silu has a slope of at most 1.1 and its own operations add less than 8 roundings
        g, u, dg, du = z[:, ::2], z[:, 1::2], t[:, ::2], t[:, 1::2]
        s = g * torch.sigmoid(g)
        z, t = s * u, 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + 8 * 2.0 ** -24 * (s * u).abs()
    check(y, z, t, "f32")


def test_many_units_of_long_rows():
    # as many tiles of rows as would be pairs of CTAs, 2,048 groups each
    rows, cols, group, m = 256 * 80 + 30, 1 << 16, 32, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    byte = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda") | 0x11
    scales = torch.full((rows, cols // group), 0.01, dtype=torch.float16, device="cuda")
    w = mm.mm_packed4(byte, scales, torch.zeros_like(scales, dtype=torch.uint8), cols, group, weights_static=True)
    torch.cuda.synchronize()
    x = torch.rand(m, cols, generator=g, device="cuda").half()
    y = torch.empty(m, rows, device="cuda")
    mm.mm_gemm_packed4(w, x, cols, m, mm.MM_ACT_NONE, y, rows)
    mm.mm_check_device_error()
    for a, b in ((0, 130), (rows // 2, rows // 2 + 300), (rows - 150, rows)):
        ref = exact(byte[a:b], scales[a:b], group, x)
        assert bool(((y[:, a:b].double() - ref).abs() <= (bound(cols, group) + 2.0 ** -24) * ref).all())


@pytest.mark.parametrize("m", [2, 40])
def test_infinities(m):
    w, byte, scales, x = same_sign("random", 1, 24, 1 << 20, 32, m, 9)
    x[1, 70000] = float("inf")
    y = torch.empty(m, 24, device="cuda")
    mm.mm_gemm_packed4(w, x, 1 << 20, m, mm.MM_ACT_NONE, y, 24)
    mm.mm_check_device_error()
    assert bool((y[1] == float("inf")).all()) and bool(y[0].isfinite().all())
