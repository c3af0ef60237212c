"""silu(gate) * up of 4-bit products: the same bits wherever Y lies, and small results of large negative gates."""
import math

import pytest
import torch

import dense_packed_bit_gb300 as mm
from packed4_util import DT, make_weights, make_x, make_y, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


@pytest.mark.parametrize("dtype,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("m,rows", [(1, 128), (13, 128), (40, 128), (130, 300), (700, 600), (300, 20480)])
def test_the_same_bits_wherever_y_lies(m, rows, dtype, out):
    w, _ = make_weights(m, 1, rows, 264, 64, dtype)
    x, _ = make_x(m + 1, m, 264, dtype)
    x *= 20  # gates of some tens
    results = []
    for pad in (8, 3, 1):  # rows of Y of whole 16 bytes, and not
        y, buf = make_y(m, rows // 2, out, pad=pad)
        mm.mm_gemm_packed4(w, x, x.stride(0), m, mm.MM_ACT_SWIGLU, y, y.stride(0))
        mm.mm_check_device_error()
        untouched(y, buf)
        results.append(y.clone())
    assert all(torch.equal(results[0], r) for r in results[1:])


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 20, 100])
def test_large_negative_gates(m, out, pad):
    """Gates of -8 s exactly, up to where exp(-gate) is still finite, and a large up-projection: within 2e-5 of itself (an
    exponential of 106 ulp, a quotient of 2, three roundings of 2^-24) and a rounding to Y's type (half a step: 2^-8)."""
    gates = [-8.0, -20.0, -64.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -1.0, 8.0, 88.0, 120.0, -0.5, -4.0, -70.0]
    n = len(gates)
    codes = torch.full((2 * n, 16), 0x88, dtype=torch.uint8)
    codes[::2, 0] = 0x80                 # column 0: 0 - 8 for the gates
    codes[1::2, 0] = 0x8C                # and 12 - 8 for the up-projections
    scales = torch.empty(2 * n, 1, dtype=torch.bfloat16)
    scales[::2, 0] = torch.tensor([-g / 8 for g in gates]).bfloat16()
    scales[1::2] = 2.0 ** 98
    assert [float(-8 * s) for s in scales[::2, 0]] == gates
    w = mm.mm_packed4(codes.cuda(), scales.cuda(), None, 32, 32)
    x = torch.zeros(m, 32, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    y, buf = make_y(m, n, out, pad=pad)
    mm.mm_gemm_packed4(w, x, 32, m, mm.MM_ACT_SWIGLU, y, y.stride(0))
    mm.mm_check_device_error()
    untouched(y, buf)
    want = torch.tensor([g / (1 + math.exp(-g)) * 2.0 ** 100 for g in gates], dtype=torch.float64)
    tol = (2e-5 + torch.finfo(DT[out]).eps / 2) * want.abs()
    assert bool(((y.double().cpu() - want).abs() <= tol).all()), (y[0].tolist(), want.tolist())
