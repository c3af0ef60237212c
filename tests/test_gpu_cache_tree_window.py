"""A tree's rows under a window whose released pages mm_cache_free has taken."""
import numpy as np
import pytest
import torch

import dense_packed_bit_gb300 as mm
from cache_util import make_cache, pack_bits, run_attention, tree_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


@pytest.mark.parametrize("n,heads", [(4, 4), (40, 4), (100, 4)])
def test_a_tree_row_without_a_bit_in_front_of_the_window(n, heads):
    # such a row sits at lens - 1 and sees the token at lens - window, which no other later query does: where
    # mm_cache_free has taken its page the call says so; with every token in place, or every row seeing itself, it does not
    lens, window, rng = [319, 300], 16, np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((2 * n, heads, 64)).astype(np.float32)).half().cuda()
    bits = [tree_bits(rng, n), tree_bits(rng, n)]
    words = -(-n // 32)
    whole = pack_bits(np.concatenate(bits), words).cuda()
    bits[0][2] = False
    empty = pack_bits(np.concatenate(bits), words).cuda()
    c, _, _ = make_cache(31, lens, [n, n], 2, 64, 16, "f16")
    run_attention(c, 0, q, [n, n], window, 0, 0.125, mask=empty)
    mm.mm_cache_free(c, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 2, window, 0)
    assert int(c.tensors[2][0, 303 // 16]) == -1
    run_attention(c, 0, q, [n, n], window, 0, 0.125, mask=whole)
    with pytest.raises(mm.MMError) as e:
        run_attention(c, 0, q, [n, n], window, 0, 0.125, mask=empty)
    assert e.value.status == mm.MM_ERR_INVALID_ARG and "out of range" in str(e.value)
