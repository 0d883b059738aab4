"""Plain 64-bit forms of the operators around a linear layer: activations and their slopes,
the int8 linear layer, rows of int8 codes, layer norm forward and backward.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the formulas that
``include/ozk.h`` states, in numpy float64; the product of the fp64 layer is
``ozaki2.dgemm``."""
from __future__ import annotations

import math

import numpy as np
from scipy import special

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C = math.sqrt(2 / math.pi)


def act(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return z * special.ndtr(z)
    if name == "gelu_tanh":
        return z * special.expit(2 * _C * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * special.expit(z)
    raise ValueError(name)


def slope(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return special.ndtr(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C * (1 + 0.134145 * z * z)
    if name == "silu":
        p = special.expit(z)
        return p * (1 + z * (1 - p))
    raise ValueError(name)


def int8_sums(x: np.ndarray, w: np.ndarray) -> np.ndarray:
    """X W^T exactly (fp64 holds every sum: |sum| <= 131071 * 2^14 < 2^53)."""
    return x.astype(np.float64) @ w.astype(np.float64).T


def int8_linear(x, sx, w, sw, bias=None, name="none", residual=None) -> np.ndarray:
    z = int8_sums(x, w) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    if bias is not None:
        z = z + bias
    c = act(z, name)
    return c if residual is None else c + residual


def layernorm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd)."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta)."""
    xh = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - xh * (g * xh).mean(1)[:, None])
    return dx, (dy * xh).sum(0), dy.sum(0)


def int8_codes(y):
    """(quotients before rounding, fp32 scale, row is all codes zero): q = rint(quotient)."""
    y = np.asarray(y, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(y).max(1)
        scale = (amax / 127.0).astype(np.float32)
        scale = np.where(np.isfinite(y).all(1) & np.isfinite(scale), scale, np.float32(np.nan))
        inv = np.where(scale > 0, 1.0 / scale.astype(np.float64), 0.0)
        quot = np.where(inv[:, None] > 0, y * inv[:, None], 0.0)
    return np.clip(quot, -127, 127), scale
