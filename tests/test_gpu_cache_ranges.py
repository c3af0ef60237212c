"""What the page calls do with values that they find out of range: the sequence (or token) is left as it was and the call
reports it."""
import numpy as np
import pytest

import dense_packed_bit_gb300 as mm
from test_gpu_cache_pages import Model, ints, reported

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def drafted():
    """Sequences of 20, 40, 0 and 0 tokens with 30, 4, 2 and 0 drafted ones in their pages."""
    m = Model(6, seqs=4, pages=30, max_pages=4, kv=1, page=16, dim=64, layers=1)
    for counts in ([20, 40, 0, 0], [30, 4, 2, 0]):
        m.reserve(counts)
        m.append(0, counts)
        if counts[1] == 40:
            m.compact(counts, [list(range(n)) for n in counts])
    return m


@pytest.mark.parametrize("with_list", [False, True])
@pytest.mark.parametrize("bad", ["starts past the tokens", "starts that fall", "more than max_new", "too many kept", "negative kept"])
def test_compact_leaves_a_sequence_out_of_range_alone(bad, with_list):
    m = drafted()
    qs, kept, tokens, most, skipped = [0, 30, 34, 36, 36], [3, 1, 2, 0], 36, 30, [0]
    if bad == "starts past the tokens":
        tokens, skipped = 33, [1, 2, 3]
    elif bad == "starts that fall":
        qs, skipped = [0, 40, 34, 36, 36], [0, 1]
    elif bad == "more than max_new":
        most = 29
    elif bad == "too many kept":
        kept[0] = 31
    else:
        kept[0] = -1
    keep = np.zeros(36, dtype=np.int32)
    for s, a in enumerate((0, 30, 34)):
        for i in range(max(0, min(kept[s], 30))):
            if a + i < 36:
                keep[a + i] = i
    mm.mm_cache_compact(m.c, ints(qs), ints(keep) if with_list else None, ints(kept), tokens, most)
    reported()
    for s in range(4):
        if s not in skipped:
            m.lens[s] += kept[s]
            m.drop(s, lambda j, s=s: j >= -(-m.lens[s] // 16))
    m.check(bad)


def test_a_list_that_does_not_rise():
    # the token that it names stays where it is, the others move, the sequence grows by all of them
    m = drafted()
    keep = np.zeros(36, dtype=np.int32)
    keep[:4] = [2, 1, 5, 7]   # the second does not rise
    keep[30:32] = [0, 9]      # the second names no new token
    keep[34:36] = [0, 1]
    before = m.k.copy(), m.v.copy()
    mm.mm_cache_compact(m.c, ints([0, 30, 34, 36, 36]), ints(keep), ints([4, 2, 2, 0]), 36, 30)
    reported()
    for i, f in ((0, 2), (2, 5), (3, 7)):
        a, b = 20 + f, 20 + i
        for pool, old in zip((m.k, m.v), before):
            pool[:, m.table[0, b // 16], :, b % 16] = old[:, m.table[0, a // 16], :, a % 16]
    for s, n in enumerate([4, 2, 2, 0]):
        m.lens[s] += n
        m.drop(s, lambda j, s=s: j >= -(-m.lens[s] // 16))
    m.check("a list that does not rise")
