"""Barriers that a whole warp has to execute together (`.aligned`: those of a cluster, and bar.sync) follow a __syncwarp in the 4-bit
products' kernels: code before them diverges -- loops whose trip counts differ by thread, a single lane's arrival -- and nothing
but a __syncwarp says that the warp is whole again."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_packed_bit_gb300", "csrc")


def statements(text):
    text = re.sub(r"//[^\n]*", "", text)
    return [s.strip() for s in re.split(r"[;{}]", text) if s.strip()]


@pytest.mark.parametrize("name,barriers", [("gemm_packed4_rows.cu", 4), ("gemm_packed4_tiles.cu", 5)])
def test_a_whole_warp_arrives(name, barriers):
    code = statements(open(os.path.join(CSRC, name)).read())
    found = 0
    for i, s in enumerate(code):
        if not re.search(r"\b(cluster_sync|bar_sync)\(", s):
            continue
        found += 1
        # fences between the two are straight-line code of the whole warp; a condition on the barrier itself is uniform
        before = [x for x in code[max(0, i - 4):i] if not x.startswith(("tc_fence", "if (cluster > 1)"))]
        assert before[-1].endswith(("__syncwarp()", "cluster_sync()")), (name, code[i - 3:i + 1])
    assert found >= barriers, found
