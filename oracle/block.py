"""Oracle of the operators around the QLoRA linear: 8-bit activation checkpoints, the
root-mean-square norm with the residual's addition, and bias / activation / residual behind the
product.  float64 throughout, except where the stored format fixes a rounding.

Pins (``tests/test_oracle_block.py``): the checkpoint format against an exact-rational search for
the scale exponent and the nearest E4M3 value; the gradients against central differences of the
forward formulas; the activations against their textbook forms at high precision points.
"""

from __future__ import annotations

import math

import numpy as np

from .nf4 import e4m3_decode, e4m3_encode_rn

GROUP = 32
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act8_quantize(x: np.ndarray):
    """x [M][K] (bf16-exact float64) -> (codes [M][ld], scale bytes [M][ceil(K / 32)]), ld = K rounded
    up to 16.  Per row and group of 32: e = the smallest integer with amax <= 448 * 2^e, clamped to
    [-117, 120]; code = E4M3 of x / 2^e, nearest even (with e = 120 at most 240, so that the value stays
    finite in bf16); a group with a non-finite value has the scale
    byte 255 (its codes are unspecified: zero here)."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    G, ld = -(-K // GROUP), -(-K // 16) * 16
    p = np.zeros((M, G * GROUP))
    p[:, :K] = x
    p = p.reshape(M, G, GROUP)
    bad = ~np.isfinite(p).all(axis=2)
    p = np.where(bad[:, :, None], 0.0, p)
    m, q = np.frexp(np.abs(p).max(axis=2))         # amax = m 2^q, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = np.where(m <= 0.875, q - 9, q - 8)
    e = np.where(m == 0, -117, np.clip(e, -117, 120))
    n = np.ldexp(p, -e[:, :, None])
    n = np.where(e[:, :, None] == 120, np.clip(n, -240.0, 240.0), n)
    codes = e4m3_encode_rn(n.astype(np.float32)).reshape(M, G * GROUP)
    out = np.zeros((M, ld), dtype=np.uint8)
    w = min(ld, G * GROUP)
    out[:, :w] = codes[:, :w]
    return out, np.where(bad, 255, e + 127).astype(np.uint8)


def act8_dequant(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """Values of a checkpoint: E4M3(code) * 2^(byte - 127); NaN for the byte 255."""
    v = np.asarray(e4m3_decode(codes[:, :K]), dtype=np.float64).reshape(codes.shape[0], K)
    e = np.repeat(scales.astype(np.int64) - 127, GROUP, axis=1)[:, :K]
    return np.where(e == 128, np.nan, np.ldexp(v, np.minimum(e, 127)))


def rmsnorm_forward(x, w, eps, residual=None) -> dict:
    """v = x + residual, rstd = 1 / sqrt(mean v^2 + eps), y = v rstd w."""
    v = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(v * v, axis=1) + eps)
    return {"v": v, "rstd": rstd, "y": v * rstd[:, None] * np.asarray(w, np.float64)}


def rmsnorm_backward(dy, h, rstd, w, dh=None) -> dict:
    """dx = dh + rstd (g - n mean(g n)), dw = sum_m dy n, with n = h rstd and g = dy w."""
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return {"dx": dx if dh is None else dx + dh, "dw": (dy * n).sum(axis=0)}


def _phi(z):
    return np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in np.ravel(z)]).reshape(np.shape(z))


def _logistic(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def act(z, name: str):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * _logistic(z)
    if name == "gelu":
        return z * _phi(z)
    if name == "gelu_tanh":
        return z * _logistic(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def act_slope(z, name: str):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = _logistic(z)
        return p + z * p * _logistic(-z)
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        v = c * (z + 0.044715 * z ** 3)
        p = _logistic(v)
        return p + z * p * _logistic(-v) * c * (1.0 + 3.0 * 0.044715 * z * z)
    return np.ones_like(z)
