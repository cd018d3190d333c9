"""The operators together as a user runs them: NormLinear's gradients against
float64 automatic differentiation of the same layer, the session's clipping,
and the example's training steps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import workloads  # noqa: E402
from oracle import operators as OO  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("tokens,d_in,d_out,block", [(96, 256, 192, 32), (77, 320, 160, 32), (200, 512, 768, 128)])
def test_layer_matches_autograd(hm, dev, tokens, d_in, d_out, block):
    """Every operand is rounded to E4M3 once (relative error at most 2^-4 per element, and at
    most 2^-10 of the largest of its block below that; about 2.6 % rms), both factors of a
    product independently: 4 % of the result's norm, doubled for the norm's
    gradient, whose input is such a product: bounds of 6 % and 8 %."""
    from head_muon_mxfp8_gb300.linear import NormLinear
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, res = rand(tokens, d_in).bfloat16(), rand(tokens, d_in).bfloat16()
    w = rand(d_out, d_in) * d_in ** -0.5
    dy, dres = rand(tokens, d_out).bfloat16(), rand(tokens, d_in).bfloat16()
    layer = NormLinear(tokens, d_in, d_out, block=block)
    layer.load_weight(w)
    layer.gamma.copy_(1 + 0.1 * rand(d_in))
    y, h = layer.forward(x, res)
    dx, dgamma = layer.backward(dy, dres)
    h64 = h.double().requires_grad_()
    w64, g64 = w.double().requires_grad_(), layer.gamma.double().requires_grad_()
    y64 = (h64 * torch.rsqrt(h64.square().mean(dim=1, keepdim=True) + 1e-5) * g64) @ w64.t()
    ((y64 * dy.double()).sum() + (h64 * dres.double()).sum()).backward()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    assert rel(y, y64.detach()) < 0.06
    assert rel(layer.g, w64.grad) < 0.06
    assert rel(dx, h64.grad) < 0.08 and rel(dgamma, g64.grad) < 0.08
    # a second backward pass adds to the main gradient
    once = layer.g.clone()
    layer.backward(dy, dres)
    assert rel(layer.g, 2 * once.double()) < 1e-6
    layer.close()
    assert hm.hm_device_error() == 0


def test_session_clip(hm, dev):
    """Ragged rank segments: the norm is of the segments alone, the canaries between them stay."""
    from head_muon_mxfp8_gb300.session import MuonSession
    cfg = workloads.get("tiny_ragged")
    data = workloads.generate(cfg, seed=3)
    s = MuonSession.from_config(cfg, device=dev)
    s.load("g", data["g"])
    norm, _ = OO.clip([data["g"]], 1.0, 1e-6)
    stats = s.clip_grad_norm(0.25 * norm).cpu().numpy()
    assert abs(stats[0] - norm) < 1e-5 * norm and abs(stats[1] - 0.25) < 1e-5
    want = data["g"] * stats[1]
    assert np.array_equal(s.fetch("g").numpy(), want)
    assert s.canary_intact()["g"]
    again = s.clip_grad_norm(10 * norm).cpu().numpy()
    assert again[1] == 1.0 and np.array_equal(s.fetch("g").numpy(), want)
    s.close()


def test_example_trains(hm, dev):
    from examples.norm_linear_step import train
    losses, stats = train(tokens=300, d_in=256, d_out=160, steps=12)
    assert losses[-1] < 0.35 * losses[0]
    assert all(np.isfinite(v).all() for v in stats)
