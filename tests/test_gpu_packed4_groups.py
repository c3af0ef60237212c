"""mm_gemm_packed4 against its definition in fp64: odd sizes, groups that the columns end in, zeros, strides, both types,
the activation, few rows and many."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import DT, check, make_weights, make_x, make_y, reference, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def product(seed, m, rows, cols, group, dtype, out, zeros=True, swiglu=False, static=False, pad=8):
    w, dense = make_weights(seed, 1, rows, cols, group, dtype, zeros, static=static)
    x, xd = make_x(seed + 1, m, cols, dtype, pad)
    y, buf = make_y(m, rows // 2 if swiglu else rows, out)
    mm.mm_gemm_packed4(w, x, x.stride(0), m, mm.MM_ACT_SWIGLU if swiglu else mm.MM_ACT_NONE, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    check(y, *reference(xd, dense[0], swiglu), out, f"{m} x {cols} to {rows}")
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 8, 9, 16, 17, 33, 130])
def test_rows(m, dtype, group):
    product(m, m, 50, 712, group, dtype, "f32")


@pytest.mark.parametrize("cols", [1, 7, 8, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 160, 255, 257, 385, 1000, 4095])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_columns(cols, group):
    for m in (1, 3, 40):
        product(cols + m, m, 19, cols, group, "f16" if cols % 2 else "bf16", "f32")


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 128, 129, 257, 1000])
def test_matrix_rows(rows):
    for m in (1, 12, 300):
        product(rows + m, m, rows, 264, 64, "bf16", "f32", zeros=False)


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("m", [1, 11, 70, 256, 257])
def test_types_and_swiglu(m, dtype, out):
    product(m, m, 90, 520, 128, dtype, out)
    product(m, m, 90, 520, 32, dtype, out, swiglu=True)
    product(m, m, 2, 520, 64, dtype, out, swiglu=True)


@pytest.mark.parametrize("m,rows,cols", [(1, 5000, 300), (1, 40, 12288), (5, 16, 12000), (16, 1536, 2048), (700, 300, 900),
                                         (1, 40000, 128), (64, 4096, 1024), (513, 1030, 2056)])
def test_larger(m, rows, cols):
    for group in (128, 32):
        product(m + group, m, rows, cols, group, "f16", "f32", static=True)


def test_the_same_call_gives_the_same_bits():
    for m in (1, 16, 200):
        a = product(5, m, 200, 3000, 64, "bf16", "f32").clone()
        for _ in range(3):
            assert torch.equal(a, product(5, m, 200, 3000, 64, "bf16", "f32"))


def test_codes_that_equal_their_zeros_give_zero():
    # the bound allows nothing else: every term is 0
    codes = torch.full((40, 512), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((40, 8), 3.0, dtype=torch.float16, device="cuda")
    w = mm.mm_packed4(codes, scales, torch.full((40, 8), 5, dtype=torch.uint8, device="cuda"), 1024, 128)
    for m in (1, 50):
        x = torch.randn(m, 1024, device="cuda").half()
        y = torch.full((m, 40), 9.0, device="cuda")
        mm.mm_gemm_packed4(w, x, 1024, m, mm.MM_ACT_NONE, y, 40)
        assert bool((y == 0).all())


def test_whole_numbers_are_exact():
    # codes, X and scales of few bits: every sum is an fp32 number
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (70, 640), generator=g, dtype=torch.uint8)
    scales = 2.0 ** torch.randint(-1, 2, (70, 40), generator=g)
    for dtype in ("f16", "bf16"):
        w = mm.mm_packed4(codes.cuda(), scales.to(DT[dtype]).cuda(), None, 1280, 32)
        code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
        for m in (1, 30, 129):
            x = torch.randint(-8, 9, (m, 1280), generator=g).double()
            y = torch.empty(m, 70, device="cuda")
            mm.mm_gemm_packed4(w, x.to(DT[dtype]).cuda(), 1280, m, mm.MM_ACT_NONE, y, 70)
            assert torch.equal(y.double().cpu(), x @ (code * scales.double().repeat_interleave(32, 1)).T)


@pytest.mark.parametrize("m", [3, 40])
def test_nan_and_infinity_stay_in_their_rows(m):
    w, dense = make_weights(3, 1, 60, 700, 64, "f16")
    x, xd = make_x(4, m, 700, "f16")
    x[1, 699] = float("nan")
    x[2, 0] = float("inf")
    y, buf = make_y(m, 60, "f32")
    mm.mm_gemm_packed4(w, x, x.stride(0), m, mm.MM_ACT_NONE, y, y.stride(0))
    untouched(y, buf)
    assert bool(y[1].isnan().all()) and bool((~y[2].isfinite()).all())
    keep = [i for i in range(m) if i not in (1, 2)]
    ref, tol = reference(xd[keep], dense[0], False)
    check(y[keep], ref, tol, "f32")


def test_largest_values():
    # 65504 x 15 x 4096 columns: far above fp16, well within fp32
    codes = torch.full((20, 2048), 0xFF, dtype=torch.uint8, device="cuda")
    w = mm.mm_packed4(codes, torch.ones(20, 32, dtype=torch.float16, device="cuda"), torch.zeros(20, 32, dtype=torch.uint8, device="cuda"), 4096, 128)
    for m in (1, 64):
        x = torch.full((m, 4096), 65504.0, dtype=torch.float16, device="cuda")
        y = torch.empty(m, 20, device="cuda")
        mm.mm_gemm_packed4(w, x, 4096, m, mm.MM_ACT_NONE, y, 20)
        want = 65504.0 * 15 * 4096
        assert bool(((y.double() - want).abs() <= 1e-5 * want).all())


def test_on_another_stream_and_captured():
    w, dense = make_weights(8, 1, 300, 1024, 128, "bf16")
    for m in (1, 90):
        x, xd = make_x(9, m, 1024, "bf16", pad=0)
        y, _ = make_y(m, 300, "f32", pad=0, rows=0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            mm.mm_gemm_packed4(w, x, 1024, m, mm.MM_ACT_NONE, y, 300)
        s.synchronize()
        ref, tol = reference(xd, dense[0], False)
        check(y, ref, tol, "f32")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                mm.mm_gemm_packed4(w, x, 1024, m, mm.MM_ACT_NONE, y, 300)
        x.copy_(x * 2)
        y.fill_(0)
        graph.replay()
        check(y, 2 * ref, 2 * tol, "f32")


def test_weights_beyond_4_gib():
    rows, cols, stride = 70000, 256, 1 << 16  # rows 64 KB apart: 4.6 GB of codes
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.empty(rows, stride, dtype=torch.uint8, device="cuda")
    codes = wide[:, :cols // 2]
    codes.copy_(torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8))
    scales = torch.full((rows, 2), 0.01, dtype=torch.float16, device="cuda")
    w = mm.mm_packed4(codes, scales, None, cols, 128)
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[-100:].double().cpu() - 8
    for m in (1, 40):
        x = torch.randn(m, cols, generator=g, device="cuda").half()
        y = torch.empty(m, rows, device="cuda")
        mm.mm_gemm_packed4(w, x, cols, m, mm.MM_ACT_NONE, y, rows)
        ref, tol = reference(x.double().cpu(), code * float(scales[0, 0]), False)
        check(y[:, -100:], ref, tol, "f32")


@pytest.mark.parametrize("static", [False, True])
@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_a_product_waits_for_the_one_whose_result_it_takes(m, static):
    """X of a call is Y of the call in front, which runs much longer: results of the time before show (each turn has other
    data, and the bits must be those of calls with the GPU waited for in between)."""
    first, _ = make_weights(1, 1, 4096, 8192, 128, "f16", static=static, spare=0)
    second, _ = make_weights(2, 1, 200, 4096, 64, "f16", static=static, spare=0)
    torch.cuda.synchronize()
    g = torch.Generator().manual_seed(m)
    xs = [torch.randn(m, 8192, generator=g).half().cuda() for _ in range(6)]
    y, z = torch.zeros(m, 4096, dtype=torch.float16, device="cuda"), torch.zeros(m, 200, device="cuda")

    def both(x, between):
        mm.mm_gemm_packed4(first, x, 8192, m, mm.MM_ACT_NONE, y, 4096)
        between()
        mm.mm_gemm_packed4(second, y, 4096, m, mm.MM_ACT_NONE, z, 200)
        between()
        return z.clone()

    want = [both(x, torch.cuda.synchronize) for x in xs]
    for _ in range(3):
        got = [both(x, lambda: None) for x in xs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
