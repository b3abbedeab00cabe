"""Rules that every kernel source keeps and that a run would show only by
chance (no GPU): what may hang or read too early is checked where it is written."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "flow_matching_dit_cosmot_b200", "csrc")


def source(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


FILES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")))


@pytest.mark.parametrize("name", FILES)
def test_no_drain_gives_up_for_a_failure_of_others(name):
    """The wait for a CTA's own copies and products in flight ends when they have landed or after its time limit,
    never because the status word holds something: mbar_wait (and warp_wait over it) returns at once then."""
    assert not re.search(r"\b(mbar_wait|warp_wait)\([^;]*Drain\)", source(name))


def test_warps_converge_before_an_aligned_cluster_barrier():
    """barrier.cluster .aligned wants every lane of the warp at the same instruction; it is issued from one place, which
    brings them together first."""
    with open(os.path.join(CSRC, "ptx.cuh"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert text.count("barrier.cluster.arrive") == 1
    assert re.search(r"void cluster_sync\(\) \{\s*__syncwarp\(\);\s*asm volatile\(\s*\"barrier\.cluster\.arrive", text)
    for name in FILES:
        assert "barrier.cluster" not in source(name)
