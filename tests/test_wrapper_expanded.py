"""Tensors whose elements share memory: the Python calls look at where a tensor's last element lies, not at how many it has (no GPU
needed: each is refused before its address is used)."""
import pytest
import torch

import dense_packed_bit_gb300 as mm
from test_abi_experts import P, f16, lib, weights, wrapped  # noqa: F401


def expanded(t, n):
    return t.expand(n, t.shape[1])


@pytest.mark.parametrize("name", ["linear", "experts"])
def test_rows_of_x_and_y(lib, name):  # noqa: F811
    def call(x, y):
        if name == "linear":
            return mm.mm_gemm_packed4(weights(), x, 200, 5, 0, y, 40, 0)
        return mm.mm_experts_gemm_packed4(weights(3), x, 200, 5, P[6], 1, P[5], 5, 0, y, 40, 0)

    wrapped(lambda: call(expanded(f16(1, 200), 5), torch.zeros(5, 40)), "X ends before")
    wrapped(lambda: call(P[3], expanded(torch.zeros(1, 40), 5)), "Y ends before")
    wrapped(lambda: call(P[3], expanded(torch.zeros(1, 40), 0)), "Y ends before")
    # a slice whose last element lies far enough is not shorter than it says
    wrapped(lambda: call(P[3], torch.zeros(5, 60)[:, :40]), "not on the GPU")


def test_logits_and_combination(lib):  # noqa: F811
    wrapped(lambda: mm.mm_experts_route(expanded(torch.zeros(1, 16), 5), 5, 16, 16, 2, 0, True, 1.0, P[1], P[2], P[3], P[4], P[5], None, 0, 0),
            "logits ends before")
    call = lambda y, r, o: mm.mm_experts_combine(y, 64, 6, P[1], P[2], 3, 2, 64, r, 64, o, 64, 0)  # noqa: E731
    wrapped(lambda: call(expanded(torch.zeros(1, 64), 6), None, f16(3, 64)), "Y ends before")


def test_tokens_of_the_cache():
    cache = mm.Cache()
    cache.head_dim, cache.dtype = 64, mm.MM_F16
    with pytest.raises(mm.MMError, match="q ends before"):
        mm._tokens(f16(1, 128).expand(5, 128), "q", cache, 5, 128, 2)
