"""Where MuonSession.clip_grad_norm takes its buffers from and on which stream it
works, on the host: allocations and calls are recorded, nothing is launched."""
import contextlib
import types
from collections import OrderedDict

import pytest

torch = pytest.importorskip("torch")

from head_muon_mxfp8_gb300 import session  # noqa: E402


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def made(monkeypatch):
    """A session without its constructor; a log of (what, current stream) in order."""
    log, current, alive = [], [_Stream(1)], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def alloc(name):
        def make(*shape, **kw):
            t = torch.zeros(*shape, dtype=kw["dtype"])
            log.append((name, current[-1].cuda_stream))
            alive.append(t)   # no address is used twice
            return t
        return make
    fake = types.SimpleNamespace(
        empty=alloc("empty"), zeros=alloc("zeros"), float32=torch.float32, uint8=torch.uint8, device=torch.device,
        cuda=types.SimpleNamespace(stream=on, current_stream=lambda *a: current[-1], Stream=_Stream))
    calls = []
    monkeypatch.setattr(session, "torch", fake)
    monkeypatch.setattr(session, "abi", types.SimpleNamespace(
        grad_list=lambda t: list(t), grad_norm_clip_workspace=lambda t: 64, HM_F32=2,
        grad_norm_clip=lambda lst, mx, eps, stats, ws, n, st: calls.append((lst, stats, ws, st))))
    s = session.MuonSession.__new__(session.MuonSession)
    s.__dict__.update(device=torch.device("cpu"), bases=[0, 96], lens=[64, 0], plan=0, chain=0,
                      g=torch.zeros(160), _clip=OrderedDict())
    return s, log, calls


def test_buffers_belong_to_the_stream_that_uses_them(made):
    s, log, calls = made
    s.clip_grad_norm(1.0, stream=_Stream(7))
    assert log and all(stream == 7 for _, stream in log)
    # nothing but the kernels writes the result: a fill would have to be ordered before them
    assert [name for name, _ in log] == ["empty", "empty"]
    assert calls[0][3] == 7


def test_streams_and_lists_do_not_share_buffers(made):
    s, log, calls = made
    a, b = [(16, 16, 4, 2)], [(4096, 4096, 4, 2)]
    for tensors in (None, a, b):
        for stream in (None, _Stream(7), _Stream(8)):
            s.clip_grad_norm(1.0, tensors=tensors, stream=stream)
    assert len({c[1] for c in calls}) == len({c[2] for c in calls}) == 9 > s.CLIP_LISTS
    assert [c[3] for c in calls] == [1, 7, 8] * 3


def test_alternating_lists_allocate_once(made):
    s, log, calls = made
    a, b = [(16, 16, 4, 2)], [(4096, 4096, 4, 2)]
    results = [s.clip_grad_norm(1.0, tensors=t) for t in (a, b) * 5]
    assert len(log) == 4 and results[0] is results[2] and results[1] is results[3] and results[0] is not results[1]
    assert [c[0] for c in calls] == [a, b] * 5


def test_kept_buffers_are_bounded(made):
    s, log, calls = made
    for k in range(40):
        s.clip_grad_norm(1.0, tensors=[(16 * k, 16 * k, 4, 2)])
    assert len(s._clip) == s.CLIP_LISTS
