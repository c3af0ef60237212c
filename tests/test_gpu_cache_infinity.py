"""An infinite value that every row sees makes its column of O infinite, not NaN: its weight is not 0 in any part of the
keys, however many parts a unit of rows is cut into."""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import DT, make_cache, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


# 256, 128 and 16 rows of one kv head; 7 to 25 blocks of 128 keys, cut into one to six parts
@pytest.mark.parametrize("new,heads", [(32, 8), (16, 8), (2, 8)])
@pytest.mark.parametrize("blocks", [7, 13, 18, 22, 25])
def test_infinite_value_in_a_late_part(blocks, new, heads):
    dtype, dim = "bf16", 64
    lens = blocks * 128 - new
    c, _, _ = make_cache(1, [lens], [new], 1, dim, 64, dtype)
    rng = np.random.default_rng(2)
    # scores within 2 of each other: every weight is far from 0
    q = torch.from_numpy((0.2 * rng.standard_normal((new, heads, dim))).astype(np.float32)).to(DT[dtype]).cuda()
    clean = run_attention(c, 0, q, [new], 0, 0, 0.125)
    _, v, table, _, _ = c.tensors
    for j in (3, lens // 2, lens - 200):  # none in the last block, which the mask cuts
        row = v[0, int(table[0, j // 64]), 0, j % 64]
        was = float(row[5])
        row[5] = float("inf")
        got = run_attention(c, 0, q, [new], 0, 0, 0.125)
        assert bool((got[..., 5] == float("inf")).all()), f"key {j}: {got[..., 5].unique().tolist()[:4]}"
        others = [x for x in range(dim) if x != 5]
        assert torch.equal(got[..., others].view(torch.int16), clean[..., others].view(torch.int16))
        row[5] = was
