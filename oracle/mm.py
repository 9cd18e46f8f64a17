"""Matrix products of MXFP4 / FP8 operands with their epilogue, and its gradient, in
float64. TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Operands are the exact values of mx.mxfp4_dequantize_values and fp8.fp8_values:
  z = A B^T + bias, d = act(z) + residual              (dense, or per expert of the rows)
  dW_e = dY_e^T X_e over the tokens of expert e         (FP8 columns, groups of 128)
  dz = act'(z) dy, db_e = column sums over expert e
Alongside each product goes `mag`, the sum of |products|, which error bounds are made of.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode
from .fp8 import fp8_scale_exponent, fp8_values
from .mx import mxfp4_dequantize_values

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


def operand_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [R, K] of (codes, E8M0 bytes) or (E4M3 bytes, fp32 scales)."""
    if scales.dtype == np.uint8:
        return mxfp4_dequantize_values(codes, scales)
    return fp8_values(codes, np.ascontiguousarray(scales, dtype=np.float32).view(np.uint32))


def sigmoid(z):
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def act(z: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0))
    if name == "gelu":
        return 0.5 * z * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * sigmoid(z)
    if name == "swiglu":
        return z[..., 0::2] * sigmoid(z[..., 0::2]) * z[..., 1::2]
    return z


def act_slope(z: np.ndarray, name: str) -> np.ndarray:
    """act'(z) elementwise (not for swiglu)."""
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        c = np.sqrt(2.0 / np.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z ** 2)
    if name == "silu":
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def act_grad(dy: np.ndarray, z: np.ndarray, name: str) -> np.ndarray:
    if name == "swiglu":
        g, u = z[..., 0::2], z[..., 1::2]
        out = np.empty_like(z)
        out[..., 0::2] = dy * u * act_slope(g, "silu")
        out[..., 1::2] = dy * g * sigmoid(g)
        return out
    return dy * act_slope(z, name)


def grouped_product(a: np.ndarray, b: np.ndarray, offsets, bias=None):
    """(z, mag) for values a [R, K], b [E, N, K], bias [E, N] and row offsets."""
    z = np.zeros((a.shape[0], b.shape[1]))
    mag = np.zeros_like(z)
    for e in range(b.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        z[r] = a[r] @ b[e].T
        mag[r] = np.abs(a[r]) @ np.abs(b[e]).T
        if bias is not None:
            z[r] += bias[e]
            mag[r] += np.abs(bias[e])
    return z, mag


def column_values(q8: np.ndarray, s_bits: np.ndarray, offsets) -> np.ndarray:
    """float64 [C, R] of FP8 columns: the experts' tokens side by side, one scale per
    128 tokens of an expert, the groups of the experts side by side."""
    R = int(offsets[-1])
    v = e4m3_decode(np.asarray(q8, dtype=np.uint8)[:, :R]).copy()
    ef = fp8_scale_exponent(s_bits)
    slot = 0
    for e in range(len(offsets) - 1):
        for t in range(int(offsets[e]), int(offsets[e + 1]), 128):
            stop = min(t + 128, int(offsets[e + 1]))
            with np.errstate(invalid="ignore"):
                v[:, t:stop] *= np.where(ef[:, slot] == 255, np.nan, np.ldexp(1.0, ef[:, slot] - 127))[:, None]
            slot += 1
    return v


def grouped_wgrad(y: np.ndarray, x: np.ndarray, offsets):
    """(d, mag) [E, N, K] for column values y [N, R], x [K, R]."""
    E = len(offsets) - 1
    d = np.zeros((E, y.shape[0], x.shape[0]))
    mag = np.zeros_like(d)
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        d[e] = y[:, r] @ x[:, r].T
        mag[e] = np.abs(y[:, r]) @ np.abs(x[:, r]).T
    return d, mag
