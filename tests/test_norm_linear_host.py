"""What NormLinear refuses, on the host: the C entry points take addresses, so a
tensor of another shape, type, layout or device has to be turned away before
any of them is called.  The binding is replaced by one that records the calls;
nothing needs a GPU."""
import types

import pytest

torch = pytest.importorskip("torch")

from head_muon_mxfp8_gb300 import linear  # noqa: E402

TOKENS, D_IN, D_OUT = 4, 64, 96
BF16 = torch.bfloat16


class _Recorder:
    """Stands in for the binding: constants by name, every other attribute a recorded call."""
    HM_F32, HM_BF16, HM_STAGE_ALL = 2, 1, 0

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args))


@pytest.fixture
def layer(monkeypatch):
    """A layer on the CPU, built without its constructor (which uploads a plan)."""
    rec = _Recorder()
    monkeypatch.setattr(linear, "abi", rec)
    monkeypatch.setattr(linear, "_stream", lambda *a: 0)
    x = linear.NormLinear.__new__(linear.NormLinear)
    x.__dict__.update(tokens=TOKENS, d_in=D_IN, d_out=D_OUT, eps=1e-5, block=32, device=torch.device("cpu"))
    mx = lambda rows, k: types.SimpleNamespace(q=torch.zeros(rows, k), s=torch.zeros(1), k=k)  # noqa: E731
    for name in ("w", "g", "_q", "_s", "_s_tiled", "gamma", "dgamma", "h", "rstd", "y", "dn", "dx", "_ws"):
        setattr(x, name, torch.zeros(D_OUT, D_IN) if name in ("w", "g") else torch.zeros(1))
    x.wt, x.x8, x.xt8, x.dy8, x.dyt8 = (mx(1, 64) for _ in range(5))
    return x, rec.calls


def _bad(rows, cols, dtype):
    """Tensors that are not [rows][cols] of `dtype`, contiguous, on the layer's device."""
    good = torch.zeros(rows, cols, dtype=dtype)
    return {
        "fewer rows": torch.zeros(rows - 1, cols, dtype=dtype),
        "more rows": torch.zeros(rows + 1, cols, dtype=dtype),
        "other width": torch.zeros(rows, cols // 2, dtype=dtype),
        "one row": torch.zeros(cols, dtype=dtype),
        "three dimensions": torch.zeros(1, rows, cols, dtype=dtype),
        "other type": torch.zeros(rows, cols, dtype=torch.float16),
        "transposed": torch.zeros(cols, rows, dtype=dtype).t(),
        "slice of wider rows": torch.zeros(rows, 2 * cols, dtype=dtype)[:, :cols],
        "expanded row": good[:1].expand(rows, cols),
        "other device": good.to("meta"),
        "no tensor": good.float().numpy(),
    }


@pytest.mark.parametrize("which", list(_bad(TOKENS, D_IN, BF16)))
@pytest.mark.parametrize("arg", ["x", "res", "dy", "dres"])
def test_activations_are_checked(layer, which, arg):
    x, calls = layer
    cols = D_OUT if arg == "dy" else D_IN
    good_in, good_out = torch.zeros(TOKENS, D_IN, dtype=BF16), torch.zeros(TOKENS, D_OUT, dtype=BF16)
    bad = _bad(TOKENS, cols, BF16)[which]
    with pytest.raises(ValueError, match=arg):
        {"x": lambda: x.forward(bad), "res": lambda: x.forward(good_in, bad), "dy": lambda: x.backward(bad),
         "dres": lambda: x.backward(good_out, bad)}[arg]()
    assert calls == []


@pytest.mark.parametrize("w", [torch.zeros(D_IN), torch.zeros(1, D_IN), torch.zeros(D_IN, D_OUT), torch.zeros(D_OUT, 1),
                               torch.zeros(())])
def test_weight_shape_is_checked(layer, w):
    x, calls = layer
    x.w.fill_(7.0)
    with pytest.raises(ValueError, match="w"):
        x.load_weight(w)
    assert calls == [] and (x.w == 7.0).all()


def test_right_tensors_are_taken(layer):
    x, calls = layer
    inp, dy = torch.zeros(TOKENS, D_IN, dtype=BF16), torch.zeros(TOKENS, D_OUT, dtype=BF16)
    x.forward(inp)
    x.forward(inp, inp)
    x.backward(dy)
    x.backward(dy, inp)
    x.load_weight(torch.zeros(D_OUT, D_IN, dtype=torch.float64))
    assert [c[0] for c in calls].count("mxfp8_gemm") == 6


def _accumulates(calls):
    return [c[1][12] for c in calls if c[0] == "rmsnorm_backward"]


def test_dgamma_adds_up_like_dw(layer, monkeypatch):
    """One step's micro-batches add to both gradients; a step, or clearing, starts both anew."""
    x, calls = layer
    x.session = types.SimpleNamespace(clip_grad_norm=lambda *a, **kw: None, run=lambda *a: None)
    x._clip = []
    monkeypatch.setattr(linear.torch.cuda, "current_stream", lambda *a: None)
    dy = torch.zeros(TOKENS, D_OUT, dtype=BF16)
    for _ in range(3):
        x.backward(dy)
    assert _accumulates(calls) == [False, True, True]
    x.step(None)
    x.backward(dy)
    x.backward(dy)
    assert _accumulates(calls)[3:] == [False, True]
    x.g.fill_(1.0)
    x.zero_grad()
    x.backward(dy)
    assert _accumulates(calls)[5:] == [False] and (x.g == 0).all()
    dw = [c[1][12] for c in calls if c[0] == "mxfp8_gemm" and c[1][11] == linear.abi.HM_F32]
    assert dw == [True] * 6


def test_every_call_runs_on_the_layers_device(layer, monkeypatch):
    """Another device being current changes nothing: launches and streams are the layer's device's."""
    x, calls = layer
    current, seen = ["another"], []

    class of:
        def __init__(self, t):
            assert t is x.gamma

        def __enter__(self):
            current.append("the layer's")

        def __exit__(self, *exc):
            current.pop()
    monkeypatch.setattr(linear.torch.cuda, "device_of", of)
    monkeypatch.setattr(linear.torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(linear, "_stream", lambda *a: seen.append(current[-1]) or 0)
    monkeypatch.setattr(type(linear.abi), "__getattr__", lambda rec, name: lambda *a: seen.append(current[-1]))
    note = lambda *a, **kw: seen.append(current[-1])  # noqa: E731
    x.session, x._clip = types.SimpleNamespace(clip_grad_norm=note, run=note), []
    inp, dy = torch.zeros(TOKENS, D_IN, dtype=BF16), torch.zeros(TOKENS, D_OUT, dtype=BF16)
    x.load_weight(torch.zeros(D_OUT, D_IN))
    x.forward(inp, inp)
    x.backward(dy, inp)
    x.step(None)
    assert len(seen) > 15 and set(seen) == {"the layer's"} and current == ["another"]
