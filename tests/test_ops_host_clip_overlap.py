"""grad_norm_clip refuses a workspace or a result inside a tensor or inside each other."""
import pytest

A, B, D, W = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(4))
N = 100_000   # elements: seven chunks of fp32, so 56 bytes of sums


def _status(hm, tensors, stats=D, ws=W):
    try:
        hm.grad_norm_clip(hm.grad_list(tensors), 1.0, 1e-6, stats, ws, 1 << 20)
    except hm.HmError as e:
        return e.status
    return 0


@pytest.mark.parametrize("tensors,kw", [
    ([(A, B, N, 2)], dict(stats=W + 16)),               # the result in the sums
    ([(A, B, N, 2)], dict(stats=A + 400)),              # ... in a source
    ([(A, B, N, 2)], dict(stats=B + 4 * N - 4)),        # ... at a destination's end
    ([(A, 0, N, 2)], dict(stats=A)),                    # ... in a tensor that is only counted
    ([(A, B, N, 2)], dict(ws=A + 4096)),                # the sums in a source
    ([(A, B, N, 2)], dict(ws=B)),
    ([(A, A, 7, 1), (B, B, N, 1)], dict(ws=B + 16)),    # ... in the second tensor
])
def test_refused(hm, tensors, kw):
    assert _status(hm, tensors, **kw) == hm.HM_ERR_OVERLAP


@pytest.mark.parametrize("tensors,kw", [
    ([(A, B, N, 2)], dict()),
    ([(A, B, N, 2)], dict(stats=A + 4 * N)),            # right behind a tensor
    ([(A, B, N, 2)], dict(stats=W + 4096)),             # behind the sums, in the rest of the workspace
    ([(A, B, N, 2), (W, W, 0, 2)], dict()),             # an empty tensor overlaps nothing
])
def test_taken(hm, tensors, kw):
    """Without a GPU the call ends at the device check, behind every argument check."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert _status(hm, tensors, **kw) in (hm.HM_ERR_ARCH, hm.HM_ERR_CUDA)
