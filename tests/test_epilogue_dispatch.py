"""The pair kernel's launcher never drops an epilogue: a tile without a kernel for it is an error.
No call reaches one (the choice of the tile knows which exist), so the launcher's own text is checked."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "head_muon_mxfp8_gb300", "csrc")


def test_a_pair_without_a_kernel_for_the_epilogue_is_an_error():
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "hm_mxgemm.cu")).read())
    body = code.split("cudaError_t launch_pair(")[1].split("\n}\n")[0]
    chosen = body.split("if constexpr (EPI == kEpiNone) {")[1].split("\n    }\n")[0]
    # after every kind that has a kernel, and before anything is launched
    assert len(re.findall(r"return launch_pair<BN, SUMS, kEpi\w+>", chosen)) == 4
    assert re.search(r"if \(p\.epilogue\) return cudaErrorInvalidValue;\s*$", chosen)
    assert "cudaLaunchKernelEx" not in body.split("if constexpr (EPI == kEpiNone) {")[0]
