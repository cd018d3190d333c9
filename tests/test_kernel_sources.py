"""Rules of the kernels' sources that no result shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "head_muon_mxfp8_gb300", "csrc")


def _code(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _starts_early(name):
    return "launch_early(" in _code(name) or "programmaticStreamSerializationAllowed" in _code(name)


EARLY = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and _starts_early(n)]


def test_files_with_early_launches():
    assert EARLY == ["hm_clip.cu", "hm_mxgemm.cu", "hm_norm.cu", "hm_quant.cu"]


@pytest.mark.parametrize("name", EARLY)
def test_no_read_only_loads_under_an_early_launch(name):
    """A kernel that starts while the one before it drains runs while that one still writes.
    Read-only loads (__ldg, ld.global.nc, what the compiler makes of a const
    __restrict__ pointer) ask for data that nobody writes during the whole kernel, so
    waiting first does not make them right."""
    found = re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", _code(name))
    assert found == []


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits_for_the_ones_before(name):
    """Each kernel of such a file waits (griddepcontrol.wait) in its body."""
    bodies = _code(name).split("__global__")[1:]
    assert bodies and all("wait_for_earlier_kernels()" in b.split("\n}\n")[0] for b in bodies)


@pytest.mark.parametrize("name", EARLY)
def test_warps_converge_before_aligned_instructions(name):
    """tcgen05.ld and the aligned cluster barriers take all lanes of a warp at the same
    instruction; after code that lanes leave at different points (a store past the last
    column, one thread's work) only a warp or block barrier brings them together."""
    lines = [x.strip() for x in _code(name).splitlines() if x.strip()]
    loose = []
    for k, line in enumerate(lines):
        if not re.match(r"(tmem_ld(16|32)|cluster_sync_all|cluster_arrive_relaxed|cluster_wait)\(", line):
            continue
        before = k - 1
        while re.match(r"(tc_fence_(before|after)\(\);|uint32_t r\[\d+\];)$", lines[before]):
            before -= 1
        if not re.match(r"(__syncwarp|__syncthreads|cluster_arrive_relaxed)\(\);$", lines[before]):
            loose.append((lines[before], line))
    assert loose == []
