"""Argument checks of the 4-bit products with group scales and of the experts' calls: each returns its status code before any
CUDA call (no GPU needed), so no pointer passed is ever dereferenced and no kernel is launched, on any machine; and what the
Python calls refuse of a tensor before its address reaches the library."""
import ctypes

import pytest
import torch

import dense_packed_bit_gb300 as mm
from dense_packed_bit_gb300 import build as mmbuild

P = [0x1000000 * (i + 1) for i in range(12)]  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    mmbuild.build()
    return mm.load_library()


def refused(lib, status):
    assert status == mm.MM_ERR_INVALID_ARG, lib.mm_last_error()
    assert lib.mm_last_error()


def weights(experts=1, **changes):
    # matrices of 40 x 200, groups of 64: rows of 112 bytes and 4 scales
    w = mm.Packed4(P[0], P[1], P[2], experts, 40, 200, 64, 112, 40 * 112, 4, 160, mm.MM_F16, 0)
    for name, value in changes.items():
        setattr(w, name, value)
    return w


BAD = [dict(codes=None), dict(scales=None), dict(codes=P[0] + 8), dict(scales=P[1] + 1), dict(experts=0), dict(experts=1025), dict(rows=0),
       dict(rows=(1 << 28) + 1), dict(cols=0), dict(cols=(1 << 28) + 1), dict(group=0), dict(group=16), dict(group=96), dict(group=256),
       dict(codes_row=96), dict(codes_row=120), dict(codes_row=-112), dict(scales_row=3), dict(dtype=mm.MM_F32), dict(dtype=-1),
       dict(weights_static=2), dict(codes_row=1 << 46), dict(scales_row=1 << 46), dict(codes_row=1 << 60), dict(codes_expert=-16),
       dict(scales_expert=-1), dict(codes_expert=1 << 60), dict(codes_expert=40 * 112 + 8), dict(codes_row=1 << 40), dict(codes_expert=1 << 40),
       dict(rows=1 << 28, scales_row=16)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_weights(lib, bad):
    w = weights(**bad)
    refused(lib, lib.mm_gemm_packed4(w, P[3], 200, 5, 0, P[4], mm.MM_F32, 40, None))
    refused(lib, lib.mm_experts_gemm_packed4(w, P[3], 200, 5, None, 1, P[5], 5, 0, P[4], mm.MM_F32, 40, None))


def test_bad_experts(lib):
    w = weights()
    w.reserved[1] = 1
    refused(lib, lib.mm_gemm_packed4(w, P[3], 200, 5, 0, P[4], mm.MM_F32, 40, None))
    refused(lib, lib.mm_gemm_packed4(None, P[3], 200, 5, 0, P[4], mm.MM_F32, 40, None))
    refused(lib, lib.mm_gemm_packed4(weights(2), P[3], 200, 5, 0, P[4], mm.MM_F32, 40, None))
    for bad in (dict(codes_expert=39 * 112), dict(scales_expert=150)):
        refused(lib, lib.mm_experts_gemm_packed4(weights(2, **bad), P[3], 200, 5, None, 1, P[5], 5, 0, P[4], mm.MM_F32, 40, None))


PRODUCT = dict(X=P[3], x_stride=200, M=5, act=0, Y=P[4], y_dtype=mm.MM_F32, y_stride=40)
BAD_PRODUCTS = [dict(X=None), dict(X=P[3] + 8), dict(x_stride=196), dict(x_stride=192), dict(x_stride=-200), dict(x_stride=(1 << 30) + 8),
                dict(M=0), dict(M=-1), dict(M=(1 << 30) + 1), dict(act=1), dict(act=3), dict(Y=None), dict(Y=P[4] + 2), dict(y_dtype=mm.MM_BF16),
                dict(y_dtype=5), dict(y_stride=39), dict(act=2, y_stride=19), dict(y_stride=-40), dict(y_stride=(1 << 30) + 1),
                dict(Y=P[3]), dict(Y=P[3] + 400), dict(Y=P[0] + 16), dict(Y=P[1] + 4), dict(Y=P[2] + 4), dict(Y=P[0] - 4 * 199)]


@pytest.mark.parametrize("bad", BAD_PRODUCTS, ids=str)
def test_bad_products(lib, bad):
    a = dict(PRODUCT, **bad)
    refused(lib, lib.mm_gemm_packed4(weights(), a["X"], a["x_stride"], a["M"], a["act"], a["Y"], a["y_dtype"], a["y_stride"], None))
    refused(lib, lib.mm_experts_gemm_packed4(weights(3), a["X"], a["x_stride"], max(a["M"], 1), P[6], 1, P[5], a["M"], a["act"], a["Y"],
                                             a["y_dtype"], a["y_stride"], None))


def test_more_units_of_work_than_32_bits(lib):
    big = dict(rows=1 << 28, codes_expert=(1 << 28) * 112, scales_expert=(1 << 28) * 4)
    refused(lib, lib.mm_experts_gemm_packed4(weights(1024, **big), P[3], 200, 5, None, 1, P[5], 5, 0, P[4], mm.MM_F32, 1 << 28, None))
    refused(lib, lib.mm_gemm_packed4(weights(rows=1 << 28), P[3], 200, 1 << 30, 0, P[4], mm.MM_F32, 1 << 28, None))


def test_swiglu_takes_pairs(lib):
    refused(lib, lib.mm_gemm_packed4(weights(rows=39), P[3], 200, 5, mm.MM_ACT_SWIGLU, P[4], mm.MM_F32, 40, None))


@pytest.mark.parametrize("x_rows,order,per_row,offsets,slots,y", [
    (4, None, 1, P[5], 5, P[4]), (5, None, 2, P[5], 5, P[4]), (0, P[6], 1, P[5], 5, P[4]), (5, P[6], 0, P[5], 5, P[4]),
    (5, P[6], (1 << 30) + 1, P[5], 5, P[4]), (5, P[6], 1, None, 5, P[4]), (5, P[6], 1, P[5] + 2, 5, P[4]), (5, P[6] + 1, 1, P[5], 5, P[4]),
    (5, P[6], 1, P[5], 0, P[4]), (5, P[6], 1, P[5], (1 << 30) + 1, P[4]), (5, P[6], 1, P[5], 5, P[6] + 16), (5, P[6], 1, P[5], 5, P[5] + 12),
    ((1 << 30) + 1, P[6], 1, P[5], 5, P[4])])
def test_bad_ragged_products(lib, x_rows, order, per_row, offsets, slots, y):
    refused(lib, lib.mm_experts_gemm_packed4(weights(3), P[3], 200, x_rows, order, per_row, offsets, slots, 0, y, mm.MM_F32, 40, None))


ROUTE = dict(logits=P[0], dtype=mm.MM_F32, tokens=300, experts=16, stride=16, top_k=2, score=0, renorm=1, scale=1.0, ids=P[1], weights=P[2],
             offsets=P[3], order=P[4], slots=P[5], workspace=P[6], workspace_bytes=1 << 20)
BAD_ROUTES = [dict(logits=None), dict(logits=P[0] + 2), dict(dtype=3), dict(dtype=-1), dict(tokens=0), dict(tokens=1 << 30), dict(experts=0),
              dict(experts=1025), dict(stride=15), dict(stride=-16), dict(stride=1 << 31), dict(top_k=0), dict(top_k=17), dict(top_k=33, experts=64, stride=64),
              dict(score=2), dict(score=-1), dict(renorm=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=None), dict(ids=P[1] + 1),
              dict(weights=None), dict(offsets=None), dict(offsets=P[3] + 2), dict(order=None), dict(slots=None), dict(workspace=None),
              dict(workspace=P[6] + 2), dict(workspace_bytes=100), dict(ids=P[0] + 400), dict(slots=P[4] + 40), dict(offsets=P[1]),
              dict(workspace=P[2]), dict(weights=P[1] + 4)]


@pytest.mark.parametrize("bad", BAD_ROUTES, ids=str)
def test_bad_routes(lib, bad):
    a = dict(ROUTE, **bad)
    refused(lib, lib.mm_experts_route(*a.values(), None))


def test_bad_route_workspaces(lib):
    n = ctypes.c_int64(-1)
    for args in ((0, 8, 2), (5, 0, 1), (5, 1025, 2), (5, 8, 0), (5, 8, 9), (5, 64, 33), (1 << 30, 8, 2)):
        refused(lib, lib.mm_experts_route_workspace(*args, ctypes.byref(n)))
    refused(lib, lib.mm_experts_route_workspace(5, 8, 2, None))
    assert mm.mm_experts_route_workspace(1, 8, 2) == 0
    assert mm.mm_experts_route_workspace(1 << 24, 32, 8) >= 0


COMBINE = dict(Y=P[0], y_dtype=mm.MM_F32, y_stride=64, y_rows=6, slots=P[1], weights=P[2], tokens=3, top_k=2, cols=64, residual=P[3],
               residual_stride=64, out=P[4], out_dtype=mm.MM_BF16, out_stride=64)
BAD_COMBINES = [dict(Y=None), dict(Y=P[0] + 2), dict(y_dtype=3), dict(out_dtype=-1), dict(y_stride=63), dict(y_stride=-64), dict(y_stride=1 << 31),
                dict(y_rows=0), dict(y_rows=1 << 31), dict(slots=None), dict(slots=P[1] + 1), dict(weights=None), dict(weights=P[2] + 2),
                dict(tokens=0), dict(tokens=1 << 30), dict(top_k=0), dict(top_k=1025), dict(cols=0), dict(cols=1 << 29), dict(residual=P[3] + 1),
                dict(residual_stride=63), dict(out=None), dict(out=P[4] + 1), dict(out_stride=63), dict(out=P[0] + 64), dict(out=P[1]),
                dict(out=P[2]), dict(out=P[3] + 64), dict(residual=P[4], residual_stride=72)]


@pytest.mark.parametrize("bad", BAD_COMBINES, ids=str)
def test_bad_combines(lib, bad):
    a = dict(COMBINE, **bad)
    refused(lib, lib.mm_experts_combine(*a.values(), None))


# ------------------------------------------------------------------ the Python calls

def wrapped(call, why):
    with pytest.raises(mm.MMError) as e:
        call()
    assert e.value.status == mm.MM_ERR_INVALID_ARG and why in str(e.value), e.value


def f16(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


X_CALLS = {
    "linear": lambda x, y: mm.mm_gemm_packed4(weights(), x, 200, 5, 0, y, 40, 0),
    "experts": lambda x, y: mm.mm_experts_gemm_packed4(weights(3), x, 200, 5, P[6], 1, P[5], 5, 0, y, 40, 0),
}


@pytest.mark.parametrize("name", X_CALLS)
def test_rows_of_x_and_y(lib, name):
    call = X_CALLS[name]
    y = torch.zeros(5, 40)
    wrapped(lambda: call(f16(5, 200).bfloat16(), y), "X must be")
    wrapped(lambda: call(f16(5, 200).float(), y), "X must be")
    wrapped(lambda: call(f16(4, 200), y), "X ends before")
    wrapped(lambda: call(f16(5, 400)[:, ::2], y), "contiguous")
    wrapped(lambda: call(f16(5, 200), y), "not on the GPU")
    wrapped(lambda: call(P[3], y.bfloat16()), "Y must be")
    wrapped(lambda: call(P[3], y[:4]), "Y ends before")
    wrapped(lambda: call(P[3], y), "not on the GPU")
    with pytest.raises(ValueError):
        call(P[3], P[4])


def test_whole_numbers(lib):
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    y, lg = torch.zeros(5, 40), torch.zeros(5, 16)
    product = lambda order, offsets: mm.mm_experts_gemm_packed4(weights(3), P[3], 200, 5, order, 1, offsets, 5, 0, y, 40, 0)  # noqa: E731
    # (Y is looked at first; give it one that passes: an address cannot be, so these stop at Y on the host)
    wrapped(lambda: product(i32(5), i32(4)), "not on the GPU")
    route = lambda **k: mm.mm_experts_route(*{**dict(logits=lg, tokens=5, experts=16, stride=16, top_k=2, score=0, renorm=True, scale=1.0,  # noqa: E731
                                                     ids=P[1], weights=P[2], offsets=P[3], order=P[4], slots=P[5]), **k}.values(), None, 0, 0)
    wrapped(lambda: route(), "not on the GPU")
    wrapped(lambda: route(logits=lg[:4]), "logits ends before")
    wrapped(lambda: route(logits=lg.double()), "logits must be")
    wrapped(lambda: route(logits=torch.zeros(5, 32)[:, ::2]), "contiguous")


def test_combine_tensors(lib):
    y, out, r = torch.zeros(6, 64), f16(3, 64), f16(3, 64)
    call = lambda **k: mm.mm_experts_combine(*{**dict(Y=y, ys=64, n=6, slots=P[1], weights=P[2], t=3, k=2, cols=64, r=r, rs=64, out=out,  # noqa: E731
                                                      os=64), **k}.values(), 0)
    wrapped(lambda: call(Y=y.double()), "Y must be")
    wrapped(lambda: call(Y=y[:5]), "Y ends before")
    wrapped(lambda: call(), "not on the GPU")


def test_packed4_tensors():
    codes, scales = torch.zeros(2, 40, 112, dtype=torch.uint8), f16(2, 40, 4)
    for bad in (dict(codes=codes.int()), dict(scales=scales.float()), dict(scales=f16(2, 40, 3)), dict(cols=225), dict(cols=0), dict(group=32),
                dict(zeros=torch.zeros(2, 40, 4)), dict(zeros=torch.zeros(2, 40, 3, dtype=torch.uint8)),
                dict(codes=torch.zeros(2, 40, 224, dtype=torch.uint8)[:, :, ::2]), dict(codes=torch.zeros(2, 40, 104, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            mm.mm_packed4(**{**dict(codes=codes, scales=scales, cols=200, group=64), **bad})
    with pytest.raises(ValueError, match="on the GPU"):
        mm.mm_packed4(codes, scales, None, 200, 64)
