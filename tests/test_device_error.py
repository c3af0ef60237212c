"""What a device error word of the 4-bit products is reported as: a bounded wait that ran out is a timeout and a range that is
wrong an invalid argument, also where both happened.  The host code compiled by itself (no GPU needed: no test makes a
kernel's wait run out); and the kernels add to their words, so that neither event replaces the other."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_packed_bit_gb300", "csrc")

PROGRAM = r"""
#include "device_error.h"
#include <cstdio>
int main() {
    for (unsigned int w = 0; w < 32; ++w) std::printf("%d ", (int)mm::device_error_status(w));
    return 0;
}
"""


def test_status_of_every_word(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()]
    ok, invalid, timeout = 0, 1, 4  # mm_status
    want = [timeout] * 32  # any code of a wait, with the bit of a range (16) or without
    want[0], want[16] = ok, invalid
    assert got == want


@pytest.mark.parametrize("kernel", ["gemm_packed4_rows.cu", "gemm_packed4_tiles.cu"])
def test_kernels_add_to_their_words(kernel):
    text = open(os.path.join(CSRC, kernel)).read()
    writes = re.findall(r"(\w+)\(&g_packed4_\w+_err", text)
    assert len(writes) >= 4 and set(writes) == {"atomicOr"}, writes
    assert not re.search(r"g_packed4_\w+_err\s*=[^=]", text)


def test_both_words_are_read_by_that_rule():
    text = open(os.path.join(CSRC, "mm_api.cu")).read()
    words = re.findall(r"const unsigned int (\w+) = mm::packed4_\w+_take_device_error", text)
    assert len(words) == 2
    for w in words:
        assert re.search(r"packed4_status\(%s\)" % w, text), w
