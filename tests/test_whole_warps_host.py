"""Warps stay together around warp-wide instructions (read from the sources: a
warp that is apart there may wait for ever, so it is never run).

A role whose lanes did different work, one lane's loop before a barrier or a
wait that some lanes gave up, meets an .aligned barrier only after __syncwarp,
and goes on from a bounded wait to warp-wide work only by a vote."""

import os
import re

import pytest

from gemm_matmulplan_broadcast_gb300.build import CSRC

BARRIER = re.compile(r'asm volatile\("(barrier\.cluster\.\w+\.\w+\.aligned|bar\.sync)')
TOGETHER = ("__syncwarp();", "__syncthreads();", "__all_sync(", "warp_wait(")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read().split("\n")


def apart(name):
    """Lines with a barrier that no statement which gathers the warp precedes
    (of the ten lines before; a barrier counts as one)."""
    lines = source(name)
    found = []
    for i, line in enumerate(lines):
        if BARRIER.search(line):
            before = lines[max(0, i - 10):i]
            if not any(any(w in b for w in TOGETHER) or BARRIER.search(b) for b in before):
                found.append("%s:%d" % (name, i + 1))
    return found


LAYERS = ["norm.cu", "score.cu", "gated.cu", "gated_few.cu", "gated_float.cu"]


@pytest.mark.parametrize("name", LAYERS)
def test_barriers_of_the_layer_plans_are_met_by_whole_warps(name):
    assert apart(name) == []


def test_score_roles_leave_their_waits_together():
    # the loading warp's one lane waits for `empty`; every other wait is a whole warp's
    text = "\n".join(source("score.cu"))
    assert re.findall(r"mbar_wait\(&sh\.(\w+)", text) == ["empty"]


@pytest.mark.parametrize("name", ["tc_ptx.cuh", "tc_gemm.cu", "fp8.cu"])
def test_barriers_of_the_matrix_tiles_are_met_by_whole_warps(name):
    assert apart(name) == []


@pytest.mark.parametrize("name", ["tc_gemm.cu", "fp8.cu"])
def test_matrix_tiles_leave_their_waits_together(name):
    # an accumulator is read by whole warps (tcgen05.ld): its wait is a vote
    assert not re.search(r"\b(mbar_wait|bar_wait)\(&s->acc_full", "\n".join(source(name)))
    # the roles of one lane meet the last barriers with the rest of their warp
    text = "\n".join(source(name))
    ends = re.findall(r"fence_before\(\);\n(.*)\n    __syncthreads\(\);\n    (?!tc_fence_after\(\);\n    const|fence_after\(\);\n    const)",
                      text)
    assert ends and all("__syncwarp();" in e for e in ends)
