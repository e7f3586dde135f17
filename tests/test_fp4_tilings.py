"""The shapes of the GPU tests reach every tiling of the products with a ring of operands that wraps."""
import os
import re

import pytest
from fp4_tilings import GEMMS, GRAMS, walk

SOURCE = os.path.join(os.path.dirname(__file__), "..", "matrix_orthogonalizing_optimizer_gb300", "csrc", "fp4_gemm.cu")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_every_tiling_wraps_its_ring(fmt):
    wraps, several = set(), set()
    for count, m, n, k, sym in [(*s, False) for s in GEMMS] + [(c, r, r, k, True) for c, r, k in GRAMS]:
        tile, slices, ring, tiles = walk(count, m, n, k, sym, fmt)
        if slices > ring:
            wraps.add(tile)
            if tiles > 1:
                several.add(tile)
    assert wraps == {(1, 64, False), (1, 128, False), (2, 192, False), (1, 128, True), (2, 256, True)}
    # tiles of 64 columns are for few tiles only, so that no group of them has a second one
    assert several == wraps - {(1, 64, False)}


def test_the_rule_is_the_librarys():
    """fp4_tilings.py restates launch_format(): these are the lines that it restates."""
    text = open(SOURCE).read()
    rule = text[text.index("int launch_format("):]
    rule = re.sub(r"\s+", " ", re.sub(r"//.*", "", rule[:rule.index("\n}\n")]))
    for line in ["m1 = up(M, 128), m2 = up(M, 256)", "single = up(p.count * (p.sym ? tri(m1) : m1 * up(N, 128)), sms)",
                 "pairs = up(p.count * (p.sym ? tri(m2) : m2 * up(N, 192)), sms / 2)",
                 "if (1.75 * (double)pairs < (double)single) return launch<FMT, 2, 256>",
                 "if (1.2 * (double)pairs < (double)single) { return launch<FMT, 2, 192>",
                 "if (2 * p.count * m1 * up(N, 128) <= sms) { return launch<FMT, 1, 64>"]:
        assert line in rule, line
    assert sorted(re.findall(r"launch<FMT, (\d), (\d+)>", rule)) == [("1", "128"), ("1", "64"), ("2", "192"), ("2", "256")]
    assert "STAGES_MAX < 8 ? STAGES_MAX : 8" in text and "MAX_SMEM = 232448" in text
