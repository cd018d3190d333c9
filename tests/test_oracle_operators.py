"""Pins of oracle.operators: automatic differentiation and differences for the
RMS norm's gradient, PyTorch's clipping, closed forms for 128-element blocks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import mxfp8 as OX  # noqa: E402
from oracle import operators as OO  # noqa: E402


@pytest.mark.parametrize("rows,d", [(1, 32), (3, 96), (7, 64)])
def test_rms_norm_and_gradient_match_autograd(rows, d):
    rng = np.random.default_rng(rows + d)
    h, dy, dres = (rng.standard_normal((rows, d)) for _ in range(3))
    gamma = 1.0 + 0.1 * rng.standard_normal(d)
    ht = torch.tensor(h, requires_grad=True)
    gt = torch.tensor(gamma, requires_grad=True)
    y = ht * torch.rsqrt(ht.square().mean(dim=1, keepdim=True) + 1e-5) * gt
    ((y * torch.tensor(dy)).sum() + (ht * torch.tensor(dres)).sum()).backward()
    rstd, y_o = OO.rms_norm(h, gamma, 1e-5)
    dx, dg = OO.rms_norm_grad(dy, h, gamma, rstd, dres)
    assert np.allclose(y_o, y.detach().numpy(), rtol=1e-13, atol=1e-13)
    assert np.allclose(dx, ht.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dg, gt.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_rms_norm_gradient_matches_differences():
    # central differences, step 1e-5: error about 1e-10 (third derivative) + 1e-16 / 1e-5 (rounding)
    rng = np.random.default_rng(3)
    h, dy = rng.standard_normal((2, 32)), rng.standard_normal((2, 32))
    gamma = 1.0 + 0.1 * rng.standard_normal(32)
    dx, dg = OO.rms_norm_grad(dy, h, gamma, OO.rms_norm(h, gamma, 1e-5)[0])
    loss = lambda hh, gg: float((OO.rms_norm(hh, gg, 1e-5)[1] * dy).sum())  # noqa: E731
    for r, c in [(0, 0), (0, 31), (1, 7), (1, 16)]:
        e = np.zeros_like(h)
        e[r, c] = 1e-5
        assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / 2e-5 - dx[r, c]) < 1e-8
        assert abs((loss(h, gamma + e[r]) - loss(h, gamma - e[r])) / 2e-5 - dg[c]) < 1e-8


@pytest.mark.parametrize("factor", [0.3, 3.0])
def test_clip_matches_torch(factor):
    rng = np.random.default_rng(9)
    grads = [rng.standard_normal(n) for n in (1, 33, 1000)]
    norm = np.sqrt(sum((g * g).sum() for g in grads))
    ps = [torch.nn.Parameter(torch.zeros(g.size, dtype=torch.float64)) for g in grads]
    for p, g in zip(ps, grads):
        p.grad = torch.tensor(g)
    got = torch.nn.utils.clip_grad_norm_(ps, norm * factor)
    o_norm, coef = OO.clip(grads, norm * factor, 1e-6)
    assert abs(o_norm - float(got)) < 1e-12 * norm
    for p, g in zip(ps, grads):
        assert np.allclose(p.grad.numpy(), g * coef, rtol=1e-12, atol=0)


def test_clip_edges():
    assert OO.clip([], 1.0, 1e-6) == (0.0, 1.0)
    assert OO.clip([np.zeros(5)], 1.0, 0.0) == (0.0, 1.0)
    n, c = OO.clip([np.array([np.inf, 1.0])], 1.0, 1e-6)
    assert n == np.inf and c == 0.0
    n, c = OO.clip([np.array([np.nan])], 1.0, 1e-6)
    assert np.isnan(n) and np.isnan(c)


def test_block_128_scale_is_the_largest_block_scale():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((5, 300)) * np.ldexp(1.0, rng.integers(-6, 7, (5, 300)))).astype(np.float32)
    q, s = OO.quantize(x, 128)
    _, s32 = OO.quantize(x, 32)
    assert q.shape == (5, 320) and s.shape == (5, 10)
    for c in range(0, 10, 4):
        assert (s[:, c:c + 4] == s32[:, c:c + 4].max(axis=1, keepdims=True)).all()
    assert (q[:, 300:] == 0).all()
    # within half a step of the value: 2^-4 relative for normal codes, 2^-10 2^e below; saturation at 448 2^e
    v = OO.dequantize(q, s)[:, :300]
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)[:, :300]
    ok = np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10)
    assert (ok | (np.abs(x) > 448 * step)).all()


def test_product_is_that_of_the_values():
    rng = np.random.default_rng(5)
    a, sa = OO.quantize(rng.standard_normal((3, 64)).astype(np.float32))
    b, sb = OO.quantize(rng.standard_normal((4, 64)).astype(np.float32))
    d, bound = OO.product(a, sa, b, sb)
    for i in range(3):
        for j in range(4):
            want = sum(OX.e4m3_decode(int(a[i, k])) * 2.0 ** (int(sa[i, k // 32]) - 127)
                       * OX.e4m3_decode(int(b[j, k])) * 2.0 ** (int(sb[j, k // 32]) - 127) for k in range(64))
            assert abs(d[i, j] - want) <= 1e-13 * bound[i, j]
