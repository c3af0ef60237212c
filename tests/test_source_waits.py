"""Waits that have a limit stand behind the wait for the kernel in front, which may run longer than the limit: in the 4-bit products a
warp that asks for static weights early fills its ring, and waits for that kernel before it waits for a free place.  The order
is read from the source: a predecessor that outlasts the limit is not something to run."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_packed_bit_gb300", "csrc")


def block(name, begin, end):
    text = open(os.path.join(CSRC, name)).read()
    assert text.count(begin) == 1, begin
    text = text[text.index(begin):]
    return text[:text.index(end)]


def test_codes_of_many_rows():
    # places are first waited for when all CRING have been asked for once, which is when `it` is CRING
    warp = block("gemm_packed4_tiles.cu", "warp == WARP_CODES) {", "warp == WARP_MMA && rank == 0")
    first = warp.index("mbar_wait")
    assert "&cempty[b]" in warp[first:first + 40]
    assert "if (it == CRING) late_wait();" in warp[:first]
    assert "++it" in warp and "if (++b == CRING) b = 0, ++use;" in warp


def test_other_roles_of_many_rows():
    text = block("gemm_packed4_tiles.cu", "const auto late_wait = [&] {", "if (CG == 1 && ksplit > 1 && warp < WARP_EPI0)")
    for role in ("warp == WARP_X && !a.order) {", "warp == WARP_MMA && rank == 0) {", "warp == WARP_MMA) {", "warp < WARP_EPI0) {",
                 '" MM_PACKED4_REGS_EPI ";'):
        part = text[text.index(role):]
        assert part.index("late_wait();") < part.index("mbar_wait"), role


def test_few_rows():
    text = block("gemm_packed4_rows.cu", "if (warp == CONSUMERS / 32) {", "template <typename T, int NT, int G>\ncudaError_t launch")
    producer, consumers = text.split("    } else {\n        const int g = lane >> 2", 1)
    for part in (producer, consumers):
        assert part.index("pdl_wait();") < part.index("mbar_wait")
