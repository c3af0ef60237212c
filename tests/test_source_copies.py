"""Bulk copies stay within their own CTA or pair: no kernel source names a bulk copy with cluster multicast, because the library is also
loaded by runs on several GPUs and a caller's tensor may lie in another GPU's memory.  (A tcgen05.commit that arrives at the
barriers of several CTAs moves no data.)"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_packed_bit_gb300", "csrc")


def statements(text):
    """Each asm statement's string literals as one text."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", text, re.S):
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))


def test_no_bulk_copy_names_multicast():
    sources = [f for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".cu", ".cuh", ".h"))]
    copies = 0
    for f in sources:
        for s in statements(open(f).read()):
            if "cp.async.bulk" in s or "cp.reduce.async.bulk" in s:
                copies += 1
                assert "multicast" not in s, (os.path.basename(f), s)
    assert copies >= 5  # the pattern finds them


def test_multicast_is_named_by_commits_only():
    for f in glob.glob(os.path.join(CSRC, "*")):
        if f.endswith((".cu", ".cuh", ".h")):
            for line in open(f):
                if ".multicast" in line:
                    assert "tcgen05.commit" in line, (os.path.basename(f), line)
