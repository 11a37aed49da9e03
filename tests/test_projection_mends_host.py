"""CPU tests of the 8-bit projections and of Muon beside test_projection_host.py: what the header says of their limits
and of what a call reads, held against the library and its sources."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "invariant_mmdit_joint_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_kernels_that_start_early_read_by_ordinary_loads():
    """A kernel behind griddepcontrol.wait is alive while the one before it writes its inputs: the language allows
    read-only loads (__ldg, ld.global.nc, const __restrict__) only for memory that nobody writes meanwhile, and the wait
    orders ordinary loads. Files with such kernels hold no read-only load."""
    early = [f for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh")) and "griddepcontrol.wait" in source(f)]
    assert {"k_fp8.cu", "k_muon.cu"} <= set(early)
    for f in early:
        found = re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__|__ldcs|__ldca", source(f))
        assert not found, (f, found)
