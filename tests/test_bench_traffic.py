"""The benchmark's DRAM bytes of a Newton-Schulz stage: reported for the workload and the
sources they were measured on, whatever the comments say, and for no others."""
import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402
import workloads  # noqa: E402


def test_reported_for_the_present_sources():
    """A change of the kernels' code calls for a new measurement (the profile of one Video-DiT layer)."""
    assert bench.ns_stage_traffic(workloads.get("video_dit")) == bench.NS_STAGE_TRAFFIC["bytes"]
    assert bench.ns_stage_traffic(workloads.get("lm_layer")) is None


@pytest.mark.parametrize("name", ["hm_ns.cu", "hm_ptx.cuh", "hm_mx_device.cuh"])
def test_code_counts_and_comments_do_not(tmp_path, name):
    for n in bench.NS_SOURCES:
        shutil.copy(os.path.join(bench.CSRC, n), tmp_path / n)
    want = bench.ns_source_hash(str(tmp_path))
    assert want == bench.ns_source_hash()
    path = tmp_path / name
    text = path.read_text()
    path.write_text("// a comment\n\n" + text.replace("\n\n", "\n\n   // another\n", 1) + "/* and\nanother */\n")
    assert bench.ns_source_hash(str(tmp_path)) == want
    path.write_text(text + "constexpr int kMore = 1;\n")
    assert bench.ns_source_hash(str(tmp_path)) != want


def test_every_file_that_the_kernels_include_counts():
    import re
    seen, todo = set(), ["hm_ns.cu"]
    while todo:
        n = todo.pop()
        if n not in seen:
            seen.add(n)
            todo += [i for i in re.findall(r'#include "([^"]+)"', open(os.path.join(bench.CSRC, n)).read())]
    # the internal header declares; device code is in the others
    assert seen - {"hm_internal.h", "hm.h"} == set(bench.NS_SOURCES)
