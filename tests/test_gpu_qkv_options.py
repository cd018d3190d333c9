"""NormQkv without the heads' norm, without rotation and with frequencies for longer
contexts, against float64 automatic differentiation of the same layer.

Bounds as test_gpu_layers.py derives them: an operand's rounding to E4M3 changes a
product by about 4 % of its norm, so q and k by 8 % at most and what takes another
product by 10 %.  What the heads' operators make of the product as it stands is off by
bf16's rounding alone, 2^-8.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
TOKENS, D, HQ, HKV, DIM = 77, 192, 3, 1, 64


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def _norm(x, gamma, eps=1e-5):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * gamma


def _frequencies(rot, theta, scaling, dev):
    """(radians per position, scale), from the definitions."""
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    s = dict(scaling or {"kind": "unscaled"})
    kind, factor = s["kind"], s.get("factor", 1.0)
    if kind == "base":
        theta *= factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "yarn":
        pair = [rot * math.log(s["trained"] / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (s["beta_fast"], s["beta_slow"])]
        low, high = max(0, math.floor(pair[0])), min(rot - 1, math.ceil(pair[1]))
        ramp = ((i - low) / (high - low)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 1 + 0.1 * math.log(factor)
    return f, 1.0


def _turn(x, positions, f, scale, rot, pairs):
    a = (positions.double()[:, None] * f)[:, None, :]
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = scale * (u * a.cos() - v * a.sin()), scale * (v * a.cos() + u * a.sin())
    return torch.cat([torch.stack([p, q], -1).flatten(-2) if pairs else torch.cat([p, q], -1), x[..., rot:]], -1)


YARN = {"kind": "yarn", "factor": 16.0, "trained": 512.0, "beta_fast": 24.0, "beta_slow": 2.0}


@pytest.mark.parametrize("norm,rot,pairs,scaling", [
    (False, 64, False, None), (False, 0, False, None), (True, 0, False, None), (False, 24, True, {"kind": "linear", "factor": 4.0}),
    (True, 64, False, YARN), (True, 32, True, {"kind": "base", "factor": 8.0}), (True, 64, False, {"kind": "unscaled"}),
], ids=str)
def test_options_match_autograd(hm, dev, norm, rot, pairs, scaling):
    from head_muon_mxfp8_gb300.layers import NormQkv
    g = torch.Generator(device=dev)
    g.manual_seed(rot + norm)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    layer = NormQkv(TOKENS, D, HQ, HKV, DIM, rot_dim=rot, pairs=pairs, theta=5e4, scaling=scaling, head_norm=norm)
    w = rand(layer.d_out, D) * D ** -0.5
    layer.load_weight(w)
    for t in (layer.gamma, layer.q_gamma, layer.k_gamma):
        t.copy_(1 + 0.1 * rand(t.numel()))
    x, dres = (rand(TOKENS, D).bfloat16() for _ in range(2))
    pos = torch.randint(0, 8000, (TOKENS,), generator=g, device=dev)
    dq, dk, dv = (rand(TOKENS, n, DIM).bfloat16() for n in (HQ, HKV, HKV))
    q, k, v, h = layer.forward(x, None, pos)
    dx, dgamma = layer.backward(dq, dk, dv, dres)
    f, scale = _frequencies(rot, 5e4, scaling, dev) if rot else (None, 1.0)
    gam = [t.double().requires_grad_() for t in (layer.gamma, layer.q_gamma, layer.k_gamma)]

    def heads(y, gamma):
        y = _norm(y, gamma) if norm else y
        return _turn(y, pos, f, scale, rot, pairs) if rot else y

    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    y = (_norm(h64, gam[0]) @ w64.t()).view(TOKENS, -1, DIM)
    q64, k64, v64 = heads(y[:, :HQ], gam[1]), heads(y[:, HQ:HQ + HKV], gam[2]), y[:, HQ + HKV:]
    ((q64 * dq.double()).sum() + (k64 * dk.double()).sum() + (v64 * dv.double()).sum() + (h64 * dres.double()).sum()).backward()
    assert torch.equal(h, x)
    assert max(_rel(q, q64.detach()), _rel(k, k64.detach()), _rel(v, v64.detach())) < 0.08
    assert _rel(layer.g, w64.grad) < 0.10 and _rel(dx, h64.grad) < 0.10 and _rel(dgamma, gam[0].grad) < 0.10
    y = layer.y.double().view(TOKENS, -1, DIM)
    for got, part, gamma in ((q, y[:, :HQ], gam[1]), (k, y[:, HQ:HQ + HKV], gam[2])):
        assert _rel(got, heads(part, gamma.detach())) < 2.0 ** -8
    grads = [layer.g, layer.dgamma]
    if norm:
        assert _rel(layer.dq_gamma, gam[1].grad) < 0.10 and _rel(layer.dk_gamma, gam[2].grad) < 0.10
        grads += [layer.dq_gamma, layer.dk_gamma]
    else:
        assert (layer.dq_gamma == 0).all() and (layer.dk_gamma == 0).all()
    once = [t.clone() for t in grads]
    layer.backward(dq, dk, dv, dres)
    assert all(_rel(t, 2 * o.double()) < 1e-6 for t, o in zip(grads, once))
    want = torch.stack([t.double().norm() for t in grads]).norm()
    stats = layer.step(hm.hm_muon_hparams(0.02, 0.9, 0.0, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, 0), max_norm=2 * float(want))
    assert abs(float(stats[0]) - float(want)) < 1e-5 * float(want) and float(stats[1]) == 1.0
    layer.close()
    assert hm.hm_device_error() == 0
