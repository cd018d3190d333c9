"""Pins of the oracle of a layer's operators: automatic differentiation and
differences in float64, PyTorch's own activations, what a rotation keeps."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import layers as OL  # noqa: E402

F = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
     "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


@pytest.mark.parametrize("name", OL.ACTS)
def test_activations_and_slopes(name):
    z = torch.linspace(-9, 9, 401, dtype=torch.float64, requires_grad=True)
    F[name](z).sum().backward()
    f, slope = OL.activate(name, z.detach().numpy())
    assert np.abs(f - F[name](z).detach().numpy()).max() < 1e-13
    assert np.abs(slope - z.grad.numpy()).max() < 1e-13
    h = 1e-6
    at = np.array([-3.1, -0.7, 0.4, 2.2])
    diff = (OL.activate(name, at + h)[0] - OL.activate(name, at - h)[0]) / (2 * h)
    assert np.abs(diff - OL.activate(name, at)[1]).max() < 1e-8


@pytest.mark.parametrize("act", OL.ACTS)
def test_epilogue_gradients_are_those_of_the_forward_forms(act):
    rng = np.random.default_rng(3)
    g, up, dd = (torch.tensor(rng.standard_normal((4, 7)), requires_grad=k < 2) for k in range(3))
    (up * F[act](g)).backward(dd)
    d_up, d_gate = OL.epilogue("gated_gradient", act, dd.numpy(), None, g.detach().numpy(), up.detach().numpy())
    assert np.allclose(d_up, up.grad.numpy(), rtol=0, atol=1e-13) and np.allclose(d_gate, g.grad.numpy(), rtol=0, atol=1e-13)
    g.grad = None
    F[act](g).backward(dd)
    assert np.allclose(OL.epilogue("gradient", act, dd.numpy(), None, g.detach().numpy())[0], g.grad.numpy(), rtol=0, atol=1e-13)
    y, z = OL.epilogue("gated", act, up.detach().numpy(), None, g.detach().numpy())
    assert np.allclose(y, (up * F[act](g)).detach().numpy(), rtol=0, atol=1e-13) and np.array_equal(z, up.detach().numpy())


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dim,rot", [(8, 8), (10, 4), (6, 0)])
def test_heads_gradient_by_differentiation_and_differences(pairs, dim, rot):
    rng = np.random.default_rng(dim + rot)
    rows, heads, eps, scale = 3, 2, 1e-3, 1.3
    ang = rng.uniform(-4, 4, (rows, rot // 2))
    x, dy, gamma = rng.standard_normal((rows, heads, dim)), rng.standard_normal((rows, heads, dim)), rng.uniform(0.5, 2, dim)
    # differentiated: real arithmetic, pair by pair
    tx, tg = torch.tensor(x, requires_grad=True), torch.tensor(gamma, requires_grad=True)
    v = tx / torch.sqrt(tx.square().mean(-1, keepdim=True) + eps) * tg
    cols = [v[..., e] for e in range(dim)]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        c, s = (torch.tensor(scale * fn(ang[:, i]))[:, None] for fn in (np.cos, np.sin))
        cols[a], cols[b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    y = torch.stack(cols, -1)
    y.backward(torch.tensor(dy))
    assert np.allclose(OL.heads(x, gamma, eps, ang, scale, pairs), y.detach().numpy(), rtol=0, atol=1e-12)
    dx, dg = OL.heads_grad(dy, x, gamma, eps, ang, scale, pairs)
    assert np.allclose(dx, tx.grad.numpy(), rtol=0, atol=1e-12) and np.allclose(dg, tg.grad.numpy(), rtol=0, atol=1e-12)
    h, e = 1e-6, np.zeros_like(x)
    e[1, 1, dim // 2] = h
    f = lambda z: float((OL.heads(z, gamma, eps, ang, scale, pairs) * dy).sum())  # noqa: E731
    assert abs((f(x + e) - f(x - e)) / (2 * h) - dx[1, 1, dim // 2]) < 1e-7
    t, none = OL.heads_grad(dy, None, None, eps, ang, scale, pairs)
    assert none is None and np.allclose(OL.turn(t, ang, 1 / scale, pairs)[..., :rot], dy[..., :rot] * 1.0, atol=1e-12)


def test_a_rotation_sees_differences_of_positions_only():
    rng = np.random.default_rng(0)
    f, _ = OL.frequencies(16, 1e4)
    q, k = rng.standard_normal((2, 1, 1, 16))
    dot = lambda m, n: float((OL.turn(q, m * f[None], 1.0, False) * OL.turn(k, n * f[None], 1.0, False)).sum())  # noqa: E731
    assert abs(dot(17, 5) - dot(1012, 1000)) < 1e-10 and abs(dot(0, 0) - float((q * k).sum())) < 1e-12


def test_frequency_scalings():
    f, _ = OL.frequencies(64, 1e4)
    assert f[0] == 1 and abs(f[-1] - 1e4 ** (-62 / 64)) < 1e-18
    b, _ = OL.frequencies(64, 1e4, "base", 8.0)
    assert abs(b[0] - 1) < 1e-15 and abs(b[-1] * 8 / f[-1] - 1) < 1e-12
    y, s = OL.frequencies(64, 1e4, "yarn", 16.0, 4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(y[turns > 40], f[turns > 40]) and np.allclose(y[turns < 0.7], f[turns < 0.7] / 16, rtol=1e-15)
    assert (np.diff(y) < 0).all() and abs(s - (1 + 0.1 * math.log(16))) < 1e-15
