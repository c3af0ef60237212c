"""The page calls at the ends of the sizes that they take."""
import pytest
import torch

import dense_packed_bit_gb300 as mm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_packed_bit_gb300 import build
    build.build()
    mm.load_library()


def test_more_pages_wanted_than_32_bits_count():
    # 128 sequences that want 2^24 pages each want 2^31 between them; 129 lack more than a whole number of 32 bits holds
    seqs, width, pages = 129, 1 << 24, 4
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")  # 8.7 GB
    k, v = (torch.zeros((1, pages, 1, 16, 8), dtype=torch.float16, device="cuda") for _ in range(2))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    need = torch.full((seqs,), 16 * width, dtype=torch.int32, device="cuda")
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n, lacking in ((2, 2 * width - pages), (127, 127 * width - pages), (128, 128 * width - pages), (129, 2 ** 31 - 1)):
        c = mm.mm_cache(k, v, table[:n], torch.zeros(n, dtype=torch.int32, device="cuda"), refs)
        mm.mm_cache_reserve(c, need, missing)
        assert missing.item() == lacking, n
        assert int(refs.sum()) == 0 and all(int(row.max()) == -1 == int(row.min()) for row in table)
    mm.mm_check_device_error()
