"""Operators of a layer's projections (oracle), float64: the product's epilogues, a
bias's gradient, norm and rotation of heads and their gradients, the rotation's
frequencies.

"SS-HSDP" trains packed QKV projections cut into heads and MLP / expert matrices
(section 3.1 EG1, Appendix A) and prints no formula for what lies between their
products.  Written here from the definitions:
    activations  max(z, 0); z Phi(z); 0.5 z (1 + tanh(sqrt(2/pi)(z + 0.044715 z^3)));
                 z / (1 + exp(-z))
    heads        v = x / sqrt(mean(x^2) + eps) * gamma, pairs of v as complex
                 numbers times scale * exp(i position freq)

Pins (tests/test_oracle_layers.py): float64 automatic differentiation and central
differences, PyTorch's activations, inner products that a rotation keeps.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_K = math.sqrt(2.0 / math.pi)
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(name, z):
    """(f(z), f'(z))."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        phi = 0.5 * _erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u, du = (z, 1.0) if name == "silu" else (2 * _K * (z + 0.044715 * z ** 3), 2 * _K * (1 + 3 * 0.044715 * z ** 2))
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-u))
    return z * s, s + z * s * (1 - s) * du


def epilogue(form, act, z, bias=None, first=None, second=None):
    """(D, out2) of the product z; first, second: the epilogue's inputs of D's shape."""
    z = np.asarray(z, dtype=np.float64)
    if bias is not None:
        z = z + np.asarray(bias, dtype=np.float64)
    if form == "forward":
        return activate(act, z)[0] + (0.0 if first is None else first), z
    f, slope = activate(act, first)
    if form == "gated":
        return z * f, z
    if form == "gradient":
        return z * slope, None
    return z * f, z * second * slope


def _pairs(rot, pairs):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)


def turn(v, angles, scale, pairs, back=False):
    """v [rows][heads][dim], angles [rows][rot / 2]."""
    rot = 2 * angles.shape[1]
    a, b = _pairs(rot, pairs)
    w = scale * np.exp(1j * (-angles if back else angles))[:, None, :]
    z = (v[..., a] + 1j * v[..., b]) * w
    out = np.array(v, dtype=np.float64)
    out[..., a], out[..., b] = z.real, z.imag
    return out


def heads(x, gamma, eps, angles, scale, pairs):
    """y of x [rows][heads][dim]; gamma None: no norm."""
    v = np.asarray(x, dtype=np.float64)
    if gamma is not None:
        v = v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * gamma
    return turn(v, angles, scale, pairs)


def heads_grad(dy, x, gamma, eps, angles, scale, pairs):
    """(dx, dgamma)."""
    t = turn(np.asarray(dy, dtype=np.float64), angles, scale, pairs, back=True)
    if gamma is None:
        return t, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    xhat, u = x * r, t * gamma
    return r * (u - xhat * np.mean(u * xhat, axis=-1, keepdims=True)), (t * xhat).sum(axis=(0, 1))


def frequencies(rot, theta, scaling="unscaled", factor=1.0, trained=1.0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of each pair, scale)."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "base":
        return (theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot), 1.0
    if scaling == "yarn":
        # pair i turns trained * theta^(-2 i / rot) / (2 pi) times: beta of them at this i
        at = [rot * math.log(trained / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (beta_fast, beta_slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0, 1)
        return f * (1 - ramp) + f / factor * ramp, 1 + 0.1 * math.log(factor)
    return f, 1.0
