"""Plain 64-bit forms of the operators of a gated feed-forward block: microscaled 4-bit lines and
the products on them, the gate and its gradient, clipping to a norm.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the formulas that
``include/ozk.h`` states, in numpy float64 and integers."""
from __future__ import annotations

import numpy as np

from . import layers

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])   # e2m1: code 0..7, sign in bit 3
BLOCK, STEP = 32, 256


def padded_k(k: int) -> int:
    return -(-k // STEP) * STEP


def mx_quant(lines: np.ndarray):
    """(codes uint8 [lines][padded k], one a byte; scales uint8 [lines][padded k / 32]).  The
    block's exponent comes from frexp (0.5 <= f < 1), a code from the midpoints between the
    grid's values, which fp64 holds: one on a midpoint takes the even code."""
    lines = np.asarray(lines, dtype=np.float64)
    n, k = lines.shape
    x = np.zeros((n, padded_k(k)))
    x[:, :k] = lines
    x = x.reshape(n, -1, BLOCK)
    amax = np.abs(x).max(2)
    finite = np.isfinite(x).all(2)
    e = np.where(amax > 0, np.frexp(np.where(finite, amax, 1.0))[1] - 1 - 2, -127)
    bad = ~finite | (e > 127)
    e = np.clip(e, -127, 127)
    v = np.abs(np.ldexp(np.where(bad[:, :, None], 0.0, x), -e[:, :, None]))
    mids = (GRID[1:] + GRID[:-1]) / 2
    below = np.searchsorted(mids, v, side="left")      # midpoints below v
    upto = np.searchsorted(mids, v, side="right")      # and those equal to it
    code = np.where((below < upto) & (below % 2 == 0), below, upto)
    code = np.where(bad[:, :, None], 0, code | np.signbit(x).astype(np.int64) << 3)
    scales = np.where(bad, 255, e + 127)
    return code.reshape(n, -1).astype(np.uint8), scales.astype(np.uint8)


def mx_pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def mx_unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def mx_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What unpacked codes and scales stand for."""
    v = np.where(codes & 8, -GRID[codes & 7], GRID[codes & 7])
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s[scales == 255] = np.nan
    return (v.reshape(v.shape[0], -1, BLOCK) * s[:, :, None]).reshape(v.shape)


def gate(z: np.ndarray, name: str) -> np.ndarray:
    """act(first half of the columns) * second half."""
    n = z.shape[1] // 2
    return layers.act(z[:, :n], name) * z[:, n:]


def gate_grad(dc: np.ndarray, z: np.ndarray, name: str) -> np.ndarray:
    """The gradient of sum(dc * gate(z))."""
    n = z.shape[1] // 2
    return np.concatenate((dc * z[:, n:] * layers.slope(z[:, :n], name),
                           dc * layers.act(z[:, :n], name)), axis=1)


def clip(tensors, max_norm: float):
    """(norm, clipped tensors); the largest magnitude is taken out before squaring."""
    flat = np.concatenate([np.asarray(t, dtype=np.float64).ravel() for t in tensors])
    most = np.abs(flat).max() if flat.size else 0.0
    if not np.isfinite(most) or most == 0:
        return (most if most == 0 else (np.nan if np.isnan(flat).any() else np.inf)), list(tensors)
    scale = 2.0 ** (np.frexp(most)[1] - 1)
    norm = float(np.sqrt(np.square(flat / scale).sum()) * scale)
    coef = max_norm / norm if norm > max_norm and np.isfinite(norm) else 1.0
    return norm, [np.asarray(t, dtype=np.float64) * coef for t in tensors]
