"""Every variant of the layer norm's gradient that is compiled is one that some
width reaches (the rule of csrc/norm.cu, restated)."""

import os
import re

from gemm_matmulplan_broadcast_gb300.build import CSRC


def columns_a_thread(pack, cols):
    """The kernel from registers: columns a thread, None where rows go elsewhere."""
    if cols > 512 * 16 or (pack > 1 and cols >= 256):
        return None
    per = 2 if pack == 1 else pack
    while per < 16 and cols > 32 * per:
        per *= 2
    return per


def test_compiled_variants_are_reached():
    reached = {(v, columns_a_thread(v, c)) for v in (1, 4, 8) for c in range(v, 9000, v)}
    reached = {(v, per // 2 if v == 1 else per // v) for v, per in reached if per}
    assert reached == {(1, 1), (1, 2), (1, 4), (1, 8), (4, 1), (4, 2), (8, 1)}
    with open(os.path.join(CSRC, "norm.cu")) as f:
        text = f.read()
    compiled = {(int(v), int(n)) for v, n in re.findall(r"backward_rows<T, (\d), (\d)>", text)}
    assert re.findall(r"backward_rows<T, V, ([^>]+)>", text) == ["V == 1 ? 4 : 8 / V"]
    assert compiled | {(1, 4), (4, 2), (8, 1)} == reached
