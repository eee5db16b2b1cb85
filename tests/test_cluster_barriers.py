"""CPU check of the sources: the aligned cluster barriers need every lane of a warp together, and lanes that took different
branches come together only where the code says so. Each one stands right behind a __syncwarp()."""
import os
import re

import pytest

from w4a4_mxfp4_quantized_b200.build import CSRC


def statements(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [line.strip() for line in text.splitlines() if line.strip()]


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_every_aligned_cluster_barrier_follows_a_syncwarp(name):
    lines = statements(name)
    for before, line in zip([""] + lines, lines):
        if "barrier.cluster." in line and ".aligned" in line:
            assert before == "__syncwarp();", f"{name}: {line}"


def test_there_are_such_barriers():
    assert any("barrier.cluster." in line for line in statements("ptx.cuh"))
