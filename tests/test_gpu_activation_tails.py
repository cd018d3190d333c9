"""Activations and slopes of the product's epilogue where they vanish, relative to the result.

The argument reaches the kernel exactly: as the bias of an empty sum (forward), or as the
gate's value beside a product of 1.  Bounds, u = 2^-24, each a sum of roundings relative to
its result:
  GELU         Phi(-|x|) = t q(t) exp(-x^2 / 2), t = 1 / (1 + p |x|): t is off by a sum's u and the
               quotient's 2^-23, which t q(t) answers with at most 2.7 times as much (0.8 / p, at 0):
               8u; Horner's last steps 3u, three products 3u, exp2's 2^-22: 18u.  The exponent: x^2, its
               product and the constant, 2.2u of x^2 / 2: 1.1 x^2 u.  For x > 0 a difference from 1: the same
               part of Phi(-x), and u.  The polynomial: fp32 2^-28, bf16 2^-13.5 (fitted to that); and half
               a bf16 step, 2^-8.
  SiLU         x / (1 + exp(-x)): the exponent's 1.3u |x|, exp2's 2^-22, the sum, the quotient's
               2^-23, the product: (1.3 |x| + 8) u.
  GELU, tanh   the same of w = x (1.6 + 0.072 x^2), which has four roundings and two
               constants': (6 |w| + 8) u.
  slopes       Phi(x) + x phi(x), s + x s (1 - s) w': both terms' bounds, of phi (1.3 x^2 + 8) u,
               w' <= 1.6 + 0.22 x^2 with 4 roundings.
Results below 2^-110, where a factor may leave the normal numbers, are bounded by that.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FIT = 2.0 ** -13.5
K = math.sqrt(2 / math.pi)


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _arguments(dev, dtype, most):
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    x = (torch.rand(4096, generator=g, device=dev, dtype=torch.float64) * 2 - 1) * most
    x[:256] = torch.linspace(-8, -3, 256, device=dev)
    x[256:288] = torch.logspace(-30, 0, 32, device=dev)
    x[288:320] = -x[256:288]
    x[320] = 0.0
    return x.to(dtype)


def _tail(x):
    return 0.5 * torch.special.erfc(x.abs() / math.sqrt(2))


def _exact(act, x):
    """(f, f', bound of f, bound of f') of x in 64 bits, for fp32 results."""
    if act == "silu":
        s = torch.sigmoid(x)
        f, rel, dw = x * s, (1.3 * x.abs() + 8) * U, 1.0
    elif act == "gelu_tanh":
        w = 2 * K * (x + 0.044715 * x ** 3)
        s, dw = torch.sigmoid(w), 2 * K * (1 + 3 * 0.044715 * x * x)
        f, rel = x * s, (6 * w.abs() + 8) * U
    else:
        p, d = 0.5 * torch.special.erfc(-x / math.sqrt(2)), torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        part = _tail(x) * (1.2 * x * x + 18) * U + p * U
        return x * p, p + x * d, x.abs() * part, part + (x * d).abs() * (1.3 * x * x + 8) * U
    slope = s + x * s * (1 - s) * dw
    # 1 - s is a difference from 1: off by s's own error and a rounding
    return f, slope, f.abs() * rel, s * rel + (f * (1 - s) * dw).abs() * (rel + 8 * U) + (f * dw).abs() * s * (rel + U)


def _bf16_more(act, x):
    """What the shorter polynomial adds to both bounds."""
    part = FIT * _tail(x) if act == "gelu" else torch.zeros_like(x)
    return x.abs() * part, part


def _near(got, want, tol, bf16):
    tol = tol + U * want.abs() + 2.0 ** -110
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(err).all()) and bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("act,most", [("gelu", 12.0), ("gelu_tanh", 8.0), ("silu", 70.0)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,pad", [(1, 0), (130, 0), (130, 3)])   # one row, whole vectors, a column per lane
def test_value_and_slope(hm, dev, act, most, out, rows, pad):
    dt, code = (torch.bfloat16, hm.HM_BF16) if out == "bf16" else (torch.float32, hm.HM_F32)
    number = {"gelu": hm.HM_ACT_GELU, "gelu_tanh": hm.HM_ACT_GELU_TANH, "silu": hm.HM_ACT_SILU}[act]
    n, ld = 4096, 4096 + pad
    a = torch.zeros(rows, 32, dtype=torch.uint8, device=dev)
    b = torch.zeros(n, 32, dtype=torch.uint8, device=dev)
    b[:, 0] = 0x38                                   # 1.0
    sa = torch.full((hm.mxfp8_tiled_scale_bytes(rows, 32),), 127, dtype=torch.uint8, device=dev)
    sb = torch.full((hm.mxfp8_tiled_scale_bytes(n, 32),), 127, dtype=torch.uint8, device=dev)
    d, gate = torch.empty(rows, ld, dtype=dt, device=dev), torch.empty(rows, ld, dtype=dt, device=dev)
    bf16 = out == "bf16"

    def call(e):
        hm.mxfp8_gemm_epilogue(a.data_ptr(), 32, sa.data_ptr(), b.data_ptr(), 32, sb.data_ptr(), rows, n, 32, d.data_ptr(), ld, code, e)
        return d[:, :n]

    x = _arguments(dev, torch.float32, most)
    f, slope, tol, tol_slope = _exact(act, x.double())
    more = _bf16_more(act, x.double()) if bf16 else (0.0, 0.0)
    _near(call(hm.hm_epilogue(hm.HM_EPI_FORWARD, number, x.data_ptr(), 0, 0, 0, 0, 0, 0)), f, tol + more[0], bf16)
    a[:, 0] = 0x38                                   # the product is 1
    x = _arguments(dev, dt, most)
    gate[:, :n] = x
    f, slope, tol, tol_slope = _exact(act, x.double())
    more = _bf16_more(act, x.double()) if bf16 else (0.0, 0.0)
    _near(call(hm.hm_epilogue(hm.HM_EPI_GATED, number, 0, gate.data_ptr(), ld, 0, 0, 0, 0)), f, tol + more[0], bf16)
    _near(call(hm.hm_epilogue(hm.HM_EPI_GRADIENT, number, 0, gate.data_ptr(), ld, 0, 0, 0, 0)), slope, tol_slope + more[1], bf16)
    assert hm.hm_device_error() == 0
