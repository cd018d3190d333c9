"""Operators around the update (oracle), float64: MXFP8 product, quantization
along either axis, RMS norm and its gradient, gradient clipping.

"SS-HSDP" section 3.1 (EG1) hands the requantized weights and their relaid-out
scales to an MXFP8 GEMM and takes a main gradient back; the paper prints no
formula for the operators in between.  Written here from their definitions:
    product   D = A B^T of the operands' dequantized values
    quantize  one UE8M0 scale per 32 (or 128) elements along an axis, G's rule
    RMS norm  h = x + r, y = h / sqrt(mean(h^2) + eps) * gamma
    clipping  g * min(1, max_norm / (norm + eps)), norm = sqrt(sum g^2)

Pins (tests/test_oracle_operators.py): float64 automatic differentiation and
central differences for the norm's gradient, PyTorch's clip_grad_norm_, and
closed forms for blocks of 128.
"""
from __future__ import annotations

import numpy as np

from . import mxfp8 as OX


def quantize(x, block=32):
    """[rows][K] float32, any K -> codes [rows][K32] and scales [rows][K32 / 32]
    (K32 = K rounded up to 32; columns past K hold zeros); block 128: one scale per
    128 columns, repeated for each 32."""
    x = np.asarray(x, dtype=np.float32)
    rows, k = x.shape
    k32 = -(-k // 32) * 32
    wide = np.zeros((rows, k32), dtype=np.float32)
    wide[:, :k] = x
    if block == 32:
        return OX.quantize_tensor(wide)
    codes = np.zeros((rows, k32), dtype=np.uint8)
    scales = np.zeros((rows, k32 // 32), dtype=np.uint8)
    for c in range(0, k32, block):
        part = wide[:, c:c + block].astype(np.float64)
        for r in range(rows):
            e = OX.scale_exponent(float(np.abs(part[r]).max()))
            codes[r, c:c + block] = OX.e4m3_encode(part[r] * 2.0 ** -e)
            scales[r, c // 32:(c + block) // 32] = e + 127
    return codes, scales


def dequantize(codes, scales):
    """float64 values of codes [rows][K] with scales [rows][K / 32]."""
    return OX.dequantize(codes.ravel(), scales.ravel()).reshape(codes.shape)


def product(a, sa, b, sb):
    """(D, bound): the product of the operands' values and the sum of the products' magnitudes."""
    x, y = dequantize(a, sa), dequantize(b, sb)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def rms_norm(h, gamma, eps):
    """(rstd, y) of float64 rows h."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return rstd, h * rstd[:, None] * np.asarray(gamma, dtype=np.float64)


def rms_norm_grad(dy, h, gamma, rstd, dres=None):
    """(dx, dgamma) from y's gradient, with rstd as the forward pass left it."""
    dy, h, gamma, rstd = (np.asarray(v, dtype=np.float64) for v in (dy, h, gamma, rstd))
    xhat = h * rstd[:, None]
    t = dy * gamma
    dx = rstd[:, None] * (t - xhat * np.mean(t * xhat, axis=1, keepdims=True))
    return dx + (0.0 if dres is None else np.asarray(dres, dtype=np.float64)), (dy * xhat).sum(axis=0)


def clip(grads, max_norm, eps):
    """(norm, coefficient) of a list of arrays."""
    with np.errstate(all="ignore"):
        norm = np.sqrt(sum((float(np.sum(np.asarray(g, dtype=np.float64) ** 2)) for g in grads), 0.0))
        c = 1.0 if norm + eps <= max_norm else np.float64(max_norm) / (norm + eps)
    return norm, c
