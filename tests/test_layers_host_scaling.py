"""A rotation's scaling that lacks what it scales by is refused, on the host and before anything
is allocated: YaRN without the trained length is plain interpolation by another name."""
import pytest

torch = pytest.importorskip("torch")

from head_muon_mxfp8_gb300 import layers  # noqa: E402


@pytest.mark.parametrize("kw", [dict(factor=16.0), {}, dict(factor=4.0, beta_fast=8.0), dict(factor=16.0, trained=None)])
def test_yarn_needs_the_trained_length(hm, kw):
    with pytest.raises(ValueError, match="trained"):
        hm.rope_turns(64, 1e4, hm.HM_ROPE_YARN, **kw)


def test_the_others_do_not(hm):
    for kind in (hm.HM_ROPE_UNSCALED, hm.HM_ROPE_LINEAR, hm.HM_ROPE_BASE):
        assert hm.rope_turns(64, 1e4, kind, factor=2.0) == hm.rope_turns(64, 1e4, kind, factor=2.0, trained=512.0)


@pytest.mark.parametrize("scaling,match", [
    ({"kind": "yarn", "factor": 16.0}, "trained"), ({"kind": "yarn", "trained": 4096.0}, "factor"), ({"kind": "linear"}, "factor"),
    ({"kind": "base", "trained": 4096.0}, "factor"), ({"factor": 8.0}, "kind"), ({"kind": "ntk", "factor": 8.0}, "kind"),
    ({"kind": "YARN", "factor": 8.0, "trained": 64.0}, "kind")])
def test_qkv_refuses_half_a_scaling(hm, monkeypatch, scaling, match):
    """Also with rot_dim = 0, where nothing would read it."""
    monkeypatch.setattr(layers.NormLinear, "__init__", lambda *a, **k: pytest.fail("allocated"))
    for rot in (None, 32, 0):
        with pytest.raises(ValueError, match=match):
            layers.NormQkv(4, 64, 2, 1, 64, rot_dim=rot, scaling=scaling, device="cpu")


@pytest.mark.parametrize("rot", [63, 66, -2])
def test_qkv_refuses_a_rotation_that_does_not_fit(hm, monkeypatch, rot):
    monkeypatch.setattr(layers.NormLinear, "__init__", lambda *a, **k: pytest.fail("allocated"))
    with pytest.raises((ValueError, hm.HmError)):
        layers.NormQkv(4, 64, 2, 1, 64, rot_dim=rot, device="cpu")
