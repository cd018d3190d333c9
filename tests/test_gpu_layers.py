"""The operators of a layer run together as a user runs them: NormQkv and NormMlp against
float64 automatic differentiation of the same layers, several passes and an update.

Bounds: an operand's rounding to E4M3 changes a product by about 4 % of its norm (both
factors rounded, 2.6 % rms each; 6 % is NormLinear's bound).  NormQkv's q and k are such a
product through a norm that keeps its size and a rotation: 8 %, its gradients another
product further, 10 %.  NormMlp: the second product's input is off by the first's 4 % times
a slope of at most 1.13 and 2.6 % for its own rounding, so its result by
sqrt(4.5^2 + 4^2) = 6 %, bound 9 %; dz is a product (4 %) times a slope taken of z that is off by 4 %
(4.5 % more where gated), dW1 and dx another product: sqrt(3) 4.5 = 8 %, bound 12 %.  Sums
over tokens (biases, gammas) average the errors of their terms: the same 12 %.  ReLU's
slope is a step: an error of 4 % of z's spread s moves E|e| phi(0) / s = 0.04 0.8 0.4 = 1.3 % of
the elements over it, half of all being on, so dz is off by sqrt(0.013 / 0.5) = 16 % from
that alone, 18 % with the rest: bound 24 %.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def _norm(x, gamma, eps=1e-5):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * gamma


def _turn(x, positions, theta, rot, pairs):
    f = theta ** (-2.0 * torch.arange(rot // 2, device=x.device, dtype=torch.float64) / rot)
    a = (positions.double()[:, None] * f)[:, None, :]
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    return torch.cat([torch.stack([p, q], -1).flatten(-2) if pairs else torch.cat([p, q], -1), x[..., rot:]], -1)


@pytest.mark.parametrize("tokens,d_in,hq,hkv,dim,rot,pairs,block", [(96, 256, 4, 2, 64, 64, False, 32), (77, 320, 2, 1, 96, 48, True, 128),
                                                                     (130, 128, 3, 1, 32, 8, False, 32)])
def test_qkv_matches_autograd(hm, dev, tokens, d_in, hq, hkv, dim, rot, pairs, block):
    from head_muon_mxfp8_gb300.layers import NormQkv
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    layer = NormQkv(tokens, d_in, hq, hkv, dim, rot_dim=rot, pairs=pairs, theta=5e4, block=block)
    w = rand(layer.d_out, d_in) * d_in ** -0.5
    layer.load_weight(w)
    for t in (layer.gamma, layer.q_gamma, layer.k_gamma):
        t.copy_(1 + 0.1 * rand(t.numel()))
    x, res, dres = (rand(tokens, d_in).bfloat16() for _ in range(3))
    pos = torch.randint(0, 100000, (tokens,), generator=g, device=dev)
    q, k, v, h = layer.forward(x, res, pos)
    # gradients as an attention hands them over: heads first
    dq, dk, dv = (rand(n, tokens, dim).bfloat16().transpose(0, 1) for n in (hq, hkv, hkv))
    dx, dgamma = layer.backward(dq, dk, dv, dres)
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    gam = [t.double().requires_grad_() for t in (layer.gamma, layer.q_gamma, layer.k_gamma)]
    y = (_norm(h64, gam[0]) @ w64.t()).view(tokens, -1, dim)
    q64 = _turn(_norm(y[:, :hq], gam[1]), pos, 5e4, rot, pairs)
    k64 = _turn(_norm(y[:, hq:hq + hkv], gam[2]), pos, 5e4, rot, pairs)
    v64 = y[:, hq + hkv:]
    ((q64 * dq.double()).sum() + (k64 * dk.double()).sum() + (v64 * dv.double()).sum() + (h64 * dres.double()).sum()).backward()
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    assert max(_rel(q, q64.detach()), _rel(k, k64.detach()), _rel(v, v64.detach())) < 0.08
    assert _rel(layer.g, w64.grad) < 0.10 and _rel(dx, h64.grad) < 0.10 and _rel(dgamma, gam[0].grad) < 0.10
    assert _rel(layer.dq_gamma, gam[1].grad) < 0.10 and _rel(layer.dk_gamma, gam[2].grad) < 0.10
    # the operators themselves, on the packed product as it is: to bf16's rounding
    y = layer.y.double().view(tokens, -1, dim)
    assert _rel(q, _turn(_norm(y[:, :hq], gam[1].detach()), pos, 5e4, rot, pairs)) < 2.0 ** -8
    # a second pass adds up
    once = [t.clone() for t in (layer.g, layer.dgamma, layer.dq_gamma, layer.dk_gamma)]
    layer.backward(dq, dk, dv, dres)
    for t, o in zip((layer.g, layer.dgamma, layer.dq_gamma, layer.dk_gamma), once):
        assert _rel(t, 2 * o.double()) < 1e-6
    # a step: the norm is of every gradient, the units are the heads
    want = torch.stack([t.double().norm() for t in (layer.g, layer.dgamma, layer.dq_gamma, layer.dk_gamma)]).norm()
    before = layer.w.clone()
    stats = layer.step(hm.hm_muon_hparams(0.02, 0.9, 0.0, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, 0), max_norm=0.5 * float(want))
    assert abs(float(stats[0]) - float(want)) < 1e-5 * float(want) and abs(float(stats[1]) - 0.5) < 1e-5
    assert layer.session.info.n_units == hq + 2 * hkv and not torch.equal(before, layer.w)
    q2, *_ = layer.forward(x, res, pos)
    assert torch.isfinite(q2.float()).all()
    layer.close()
    assert hm.hm_device_error() == 0


ACT = {"gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"), "gelu": torch.nn.functional.gelu,
       "silu": torch.nn.functional.silu, "relu": torch.relu}


@pytest.mark.parametrize("tokens,d,ff,act,gated,bias,block", [(96, 256, 512, "gelu_tanh", False, True, 32), (77, 160, 320, "silu", True, False, 32),
                                                               (200, 128, 384, "gelu", True, True, 128), (33, 64, 96, "relu", False, False, 32)])
def test_mlp_matches_autograd(hm, dev, tokens, d, ff, act, gated, bias, block):
    from head_muon_mxfp8_gb300.layers import NormMlp
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    layer = NormMlp(tokens, d, ff, activation=act, gated=gated, bias=bias, block=block)
    ws = [rand(ff, d) * d ** -0.5 for _ in range(1 + gated)] + [rand(d, ff) * ff ** -0.5]
    layer.load_weights(*ws)
    layer.gamma.copy_(1 + 0.1 * rand(d))
    for b in layer.biases:
        if b is not None:
            b.copy_(0.3 * rand(b.numel()))
    x, res, dy = (rand(tokens, d).bfloat16() for _ in range(3))
    y, h = layer.forward(x, res)
    dx, dgamma = layer.backward(dy)
    h64, g64 = h.double().requires_grad_(), layer.gamma.double().requires_grad_()
    w64 = [w.double().requires_grad_() for w in ws]
    b64 = [b.double().requires_grad_() if b is not None else torch.zeros((), device=dev) for b in layer.biases]
    n = _norm(h64, g64)
    z = [n @ w.t() + b for w, b in zip(w64[:-1], b64[:-1])]
    a = ACT[act](z[0]) * z[1] if gated else ACT[act](z[0])
    mlp = a @ w64[-1].t() + b64[-1]
    ((h64 + mlp) * dy.double()).sum().backward()
    assert _rel(y.double() - h.double(), mlp.detach()) < 0.09 + 2.0 ** -8 * float(y.double().norm() / mlp.detach().norm())
    most = 0.24 if act == "relu" else 0.12
    assert all(_rel(w.g, r.grad) < most for w, r in zip(layer.weights, w64))
    assert _rel(dx, h64.grad) < most and _rel(dgamma, g64.grad) < most
    if bias:
        assert all(_rel(b, r.grad) < most for b, r in zip(layer.dbiases, b64))
        want = dy.double().sum(dim=0)   # the last bias's gradient is dy's own sum
        assert _rel(layer.dbiases[-1], want) < 1e-6
    small = [layer.dgamma] + [b for b in layer.dbiases if b is not None]
    once = [t.clone() for t in [w.g for w in layer.weights] + small]
    layer.backward(dy)
    for t, o in zip([w.g for w in layer.weights] + small, once):
        assert _rel(t, 2 * o.double()) < 1e-6
    want = torch.stack([t.double().norm() for t in [w.g for w in layer.weights] + small]).norm()
    stats = layer.step(hm.hm_muon_hparams(0.02, 0.9, 0.0, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, 0), max_norm=10 * float(want))
    assert abs(float(stats[0]) - float(want)) < 1e-5 * float(want) and float(stats[1]) == 1.0
    assert all(not torch.equal(w.w, t) for w, t in zip(layer.weights, ws))
    y2, _ = layer.forward(x, res)
    assert torch.isfinite(y2.float()).all() and not torch.equal(y2, layer.h)
    layer.close()
    assert hm.hm_device_error() == 0


def _passes(dev, which, tokens):
    """A layer, its inputs and one training pass over them -> the results, copied."""
    from head_muon_mxfp8_gb300.layers import NormMlp, NormQkv
    g = torch.Generator(device=dev)
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if which == "qkv":
        layer = NormQkv(tokens, 160, 3, 1, 64, rot_dim=32)
        layer.load_weight(rand(layer.d_out, 160) * 160 ** -0.5)
        inputs = [rand(tokens, 160).bfloat16(), rand(tokens, 160).bfloat16(), torch.randint(0, 5000, (tokens,), generator=g, device=dev)]
        inputs += [rand(tokens, n, 64).bfloat16() for n in (3, 1, 1)]
    else:
        layer = NormMlp(tokens, 160, 352, activation="silu", gated=True)
        layer.load_weights(*[rand(*s) * 0.07 for s in ((352, 160), (352, 160), (160, 352))])
        inputs = [rand(tokens, 160).bfloat16() for _ in range(3)]

    def one():
        layer.zero_grad()
        if which == "qkv":
            outs = [*layer.forward(*inputs[:3]), *layer.backward(*inputs[3:])]
            return outs + [layer.g, layer.dq_gamma, layer.dk_gamma]
        return [*layer.forward(*inputs[:2]), *layer.backward(inputs[2]), layer.session.g, *layer.dbiases]
    return layer, inputs, one


@pytest.mark.parametrize("which,tokens", [("qkv", 1), ("qkv", 77), ("mlp", 1), ("mlp", 77)])
def test_captured_passes_repeat_eager_ones(hm, dev, which, tokens):
    """A graph of a whole pass, the layer's first backward pass in it, replayed on new inputs:
    bit for bit the eager pass on those inputs, before and after it."""
    layer, inputs, one = _passes(dev, which, tokens)
    other, theirs, eager = _passes(dev, which, tokens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = one()
    for _ in range(2):
        for t, o in zip(inputs, theirs):
            t.copy_(t.flip(0) if t.dtype == torch.int64 else t * -0.75)
            o.copy_(t)
        want = [t.clone() for t in eager()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(one(), want))
    layer.close()
    other.close()
    assert hm.hm_device_error() == 0
