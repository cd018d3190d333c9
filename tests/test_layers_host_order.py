"""NormMlp's backward pass needs a forward pass before it: what it reads would be what the buffers
were allocated with.  On the host, with a binding that records the calls."""
import types

import pytest

torch = pytest.importorskip("torch")

from head_muon_mxfp8_gb300 import layers  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Recorder:
        HM_F32, HM_BF16, HM_ACT_NONE = 2, 1, 0
        HM_EPI_FORWARD, HM_EPI_GATED, HM_EPI_GRADIENT, HM_EPI_GATED_GRADIENT = range(4)
        fails = None

        def __getattr__(self, name):
            def call(*args):
                made.append(name)
                if name == self.fails:
                    raise RuntimeError(name)
                return 64 if name.endswith("workspace") else []
            return call

    r = Recorder()
    monkeypatch.setattr(layers, "abi", r)
    monkeypatch.setattr(layers, "_stream", lambda *a: 0)
    return r, made


@pytest.fixture(params=[False, True], ids=["plain", "gated"])
def layer(calls, monkeypatch, request):
    class Session:
        def __init__(self, n, units, **kw):
            self.bases, self.w, self.g, self.m = [0], torch.zeros(n), torch.zeros(n), torch.zeros(n)
            self.q, self.s = torch.zeros(n, dtype=torch.uint8), torch.zeros(n // 32, dtype=torch.uint8)

        def grad_list(self):
            return []

    monkeypatch.setattr(layers, "MuonSession", Session)
    monkeypatch.setattr(layers, "MxBuffer", lambda rows, k, dev: types.SimpleNamespace(q=torch.zeros(1), s=torch.zeros(1), k=k))
    monkeypatch.setattr(layers._Weight, "__init__", lambda w, session, offset, rows, cols, dev: w.__dict__.update(
        rows=rows, cols=cols, g=torch.zeros(1), q=torch.zeros(1), s_tiled=torch.zeros(1), t=types.SimpleNamespace(q=torch.zeros(1), s=torch.zeros(1), k=cols)))
    monkeypatch.setattr(layers, "ACTIVATIONS", {"none": 0})
    x = layers.NormMlp(4, 64, 96, activation="none", gated=request.param, device="cpu")
    calls[1].clear()
    return x


def test_backward_needs_a_forward_pass(calls, layer):
    rec, made = calls
    x = dy = torch.zeros(4, 64, dtype=BF16)
    with pytest.raises(ValueError, match="forward"):
        layer.backward(dy)
    assert made == [] and not layer._summed
    layer.forward(x)
    made.clear()
    layer.backward(dy)
    layer.backward(dy)   # another micro-batch's gradient of the same pass
    assert made.count("rmsnorm_backward") == 2


def test_a_forward_pass_that_stopped_half_way_is_none(calls, layer):
    rec, made = calls
    x = dy = torch.zeros(4, 64, dtype=BF16)
    layer.forward(x)
    rec.fails = "mxfp8_quantize"   # after the first products
    with pytest.raises(RuntimeError):
        layer.forward(x)
    rec.fails = None
    made.clear()
    with pytest.raises(ValueError, match="forward"):
        layer.backward(dy)
    assert made == []
    # a refused input leaves the pass before as it was
    layer.forward(x)
    with pytest.raises(ValueError):
        layer.forward(x.float())
    layer.backward(dy)
    assert made[-1] == "rmsnorm_backward"
