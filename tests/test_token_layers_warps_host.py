"""Warps stay together around warp-wide instructions in the kernels of the
residual norm, sampling and embedding plans (as in test_whole_warps_host.py)."""

import pytest

from test_whole_warps_host import apart, source


@pytest.mark.parametrize("name", ["residual.cu", "sample.cu", "embedding.cu"])
def test_barriers_are_met_by_whole_warps(name):
    assert apart(name) == []


def test_waits_have_a_limit():
    # the one kernel that waits for copies leaves its waits by the bounded form, and drains what it asked for
    text = "\n".join(source("residual.cu"))
    assert text.count("tc::mbar_wait(") == 1 and text.count("tc::mbar_wait_drain(") == 2 and "try_wait" not in text
    assert "mbar" not in "\n".join(source("sample.cu")) + "\n".join(source("embedding.cu"))
