"""Routing with logits of +infinity: they are picked first, softmax weights of their tokens are NaN, and their sigmoid is 1."""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from test_gpu_experts import route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


INF = float("inf")
ROWS = [[1.0, INF, 0.0, -INF], [INF, -2.0, INF, INF], [0.5, -1.0, 2.0, 0.0], [-INF, -INF, INF, float("nan")]]
PICKS = [[1, 0, 2], [0, 2, 3], [2, 0, 3], [2, -1, -1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("repeat", [1, 30])
@pytest.mark.parametrize("renorm", [False, True])
def test_infinite_logits(renorm, repeat, dtype):
    x = torch.tensor(ROWS * repeat, device="cuda").to(dtype)
    ids, w, *_ = route(x, 3, mm.MM_ROUTE_SIGMOID, renorm)
    assert ids.tolist() == PICKS * repeat
    score = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
    with np.errstate(over="ignore"):
        want = np.array([[score(ROWS[i][p]) if p >= 0 else 0 for p in PICKS[i]] for i in range(4)] * repeat)
    if renorm:
        want = want / want.sum(1, keepdims=True)
    assert np.all(np.abs(w - want) <= 1e-5 * want)  # an exponential, a quotient and the sum: a few roundings
    ids, w, *_ = route(x, 3, mm.MM_ROUTE_SOFTMAX, renorm)
    assert ids.tolist() == PICKS * repeat
    nan = np.isnan(w).reshape(repeat, 4, 3)
    for i in range(4):
        infinite = any(v == INF for v in ROWS[i])
        assert bool((nan[:, i] == (infinite & (np.array(PICKS[i]) >= 0))).all())
