"""What NormQkv and NormMlp refuse, on the host, before any C entry point is called; the
binding is replaced by one that records the calls, nothing needs a GPU."""
import types

import pytest

torch = pytest.importorskip("torch")

from head_muon_mxfp8_gb300 import layers, linear  # noqa: E402

BF16 = torch.bfloat16


class _Recorder:
    HM_F32, HM_BF16, HM_ROPE_HALF = 2, 1, 0
    HM_EPI_FORWARD = HM_EPI_GATED = HM_EPI_GRADIENT = HM_EPI_GATED_GRADIENT = HM_ACT_NONE = 0

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 64 if name.endswith("workspace") else []
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    for m in (layers, linear):
        monkeypatch.setattr(m, "abi", r)
        monkeypatch.setattr(m, "_stream", lambda *a: 0)
    return r


def _mx(k=64):
    return types.SimpleNamespace(q=torch.zeros(1), s=torch.zeros(1), k=k)


@pytest.fixture
def qkv(rec):
    x = layers.NormQkv.__new__(layers.NormQkv)
    x.__dict__.update(tokens=4, d_in=64, d_out=4 * 32, q_heads=2, kv_heads=1, head_dim=32, head_norm=True, eps=1e-5, block=32,
                      device=torch.device("cpu"), _rot=(1.0, 32, 0), _positions=None, _head_ws=None)
    for name in ("w", "g", "_q", "_s", "_s_tiled", "gamma", "dgamma", "h", "rstd", "dn", "dx", "_ws", "_turns", "q_gamma", "k_gamma",
                 "dq_gamma", "dk_gamma"):
        setattr(x, name, torch.zeros(1))
    x.y, x._dy = torch.zeros(4, 128, dtype=BF16), torch.zeros(4, 128, dtype=BF16)
    x.q, x.k = torch.zeros(4, 2, 32, dtype=BF16), torch.zeros(4, 1, 32, dtype=BF16)
    x.wt, x.x8, x.xt8, x.dy8, x.dyt8 = (_mx() for _ in range(5))
    return x


def test_qkv_refusals(rec, qkv):
    x, pos = torch.zeros(4, 64, dtype=BF16), torch.zeros(4, dtype=torch.int64)
    dq, dk = torch.zeros(4, 2, 32, dtype=BF16), torch.zeros(4, 1, 32, dtype=BF16)
    with pytest.raises(ValueError, match="forward"):
        qkv.backward(dq, dk, dk)
    for bad in (pos[:3], pos.int(), pos.float(), pos.view(2, 2), torch.zeros(8, dtype=torch.int64)[::2], [0, 1, 2, 3], pos.to("meta")):
        with pytest.raises(ValueError, match="positions"):
            qkv.forward(x, None, bad)
    with pytest.raises(ValueError, match="x"):
        qkv.forward(x.float(), None, pos)
    assert rec.calls == []
    qkv.forward(x, None, pos)
    assert rec.calls[-1] == "head_norm_rope" and "mxfp8_gemm" in rec.calls
    rec.calls.clear()
    wrong = [dq[:3], dq.float(), dq[..., :16], dq.transpose(1, 2), dq[:, :1], dq.to("meta"), None, torch.zeros(4, 2, 64, dtype=BF16)[..., ::2]]
    for bad in wrong:
        with pytest.raises(ValueError, match="dq"):
            qkv.backward(bad, dk, dk)
    for args, name in (((dq, dq, dk), "dk"), ((dq, dk, dq), "dv")):
        with pytest.raises(ValueError, match=name):
            qkv.backward(*args)
    with pytest.raises(ValueError, match="dres"):
        qkv.backward(dq, dk, dk, x.float())
    assert rec.calls == []
    heads_first = torch.zeros(2, 4, 32, dtype=BF16).transpose(0, 1)
    qkv.backward(heads_first, dk, dk.expand(4, 1, 32))
    assert "head_norm_rope_backward" in rec.calls and rec.calls[-1] == "rmsnorm_backward"


def test_mlp_refusals(rec):
    with pytest.raises(ValueError, match="32"):
        layers.NormMlp(4, 60, 64)
    with pytest.raises(ValueError, match="activation"):
        layers.NormMlp(4, 64, 64, activation="tanh")
    x = layers.NormMlp.__new__(layers.NormMlp)
    x.__dict__.update(tokens=4, d=64, d_ff=96, gated=False, device=torch.device("cpu"), gamma=torch.zeros(64), weights=[1, 2])
    good = torch.zeros(4, 64, dtype=BF16)
    for bad in (good[:3], good.float(), good.t(), torch.zeros(4, 128, dtype=BF16)[:, :64], good.to("meta"), None):
        for call in (lambda t: x.forward(t), lambda t: x.backward(t)):
            with pytest.raises(ValueError):
                call(bad)
    with pytest.raises(ValueError, match="res"):
        x.forward(good, good[:2])
    with pytest.raises(ValueError, match="matrices"):
        x.load_weights(torch.zeros(96, 64))
    assert rec.calls == []
