"""The device headers follow the rules of the kernels that include them: code that runs
while the kernel before still writes makes no read-only loads, and nothing divides
lanes of a warp from a barrier that it shares."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "head_muon_mxfp8_gb300", "csrc")
HEADERS = sorted(n for n in os.listdir(CSRC) if n.endswith(".cuh"))


def _code(name):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)


@pytest.mark.parametrize("name", HEADERS)
def test_no_read_only_loads(name):
    assert re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", _code(name)) == []


def test_pieces_converge_before_they_turn():
    """Both barriers of a piece's way through shared memory come before any lane can leave."""
    body = _code("hm_epilogue.cuh").split("void finish(const MxGemmArgs& p, float* stage")[1]
    first, second = (m.start() for m in list(re.finditer(r"__syncwarp\(\)", body))[:2])
    assert body[:second].count("return") == 0 and first < second
