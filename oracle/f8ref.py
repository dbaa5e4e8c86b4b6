"""Plain NumPy oracle of the 8-bit floating-point operators (E4M3 codes with an
fp32 scale for blocks of 128) and of the gated feed-forward block on them, in 64
bits and without the library's code.

Codes are uint8 [R, K]; scales are float32 [ceil(R/block), ceil(K/128)], block
1 or 128."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

TOP, LOWEST = 448.0, 2.0 ** -100


def code_value(b):
    """The value of code b as a Fraction (None for the two NaN codes): sign,
    four exponent bits (bias 7), three mantissa bits, the exponent 0 subnormal."""
    ex, man = (b >> 3) & 15, b & 7
    if ex == 15 and man == 7:
        return None
    v = Fraction(man, 512) if ex == 0 else Fraction(8 + man) * Fraction(2) ** (ex - 10)
    return -v if b & 128 else v


VALUES = np.array([np.nan if code_value(b) is None else float(code_value(b)) for b in range(256)])
VALUES[128] = -0.0


def f8_quantize(x, block=1, transpose=False):
    """(codes, scales) of x [M, K] by the definition.  The quotient 448 v / A
    has its one rounding at 2^-53: a middle between two codes is exact, and
    other quotients of fp32 numbers are at least 2^-30 away from one."""
    x = np.asarray(x, dtype=np.float64)
    if transpose:
        x = np.concatenate([x, np.zeros((-x.shape[0] % 16, x.shape[1]))]).T
    R, K = x.shape
    rows, cols = -(-R // block), -(-K // 128)
    p = np.zeros((rows * block, cols * 128))
    p[:R, :K] = x
    p = p.reshape(rows, block, cols, 128)
    finite = np.isfinite(p).all(axis=(1, 3))
    a = np.maximum(np.where(finite[:, None, :, None], np.abs(p), 0.0).max(axis=(1, 3)), LOWEST)
    q = np.where(finite[:, None, :, None], np.abs(p) * TOP / a[:, None, :, None], 0.0)
    grid = VALUES[:127]
    low = np.clip(np.searchsorted(grid, q, side="right") - 1, 0, 125)
    down, up = q - grid[low], grid[low + 1] - q
    code = np.where((down < up) | ((down == up) & (low % 2 == 0)), low, low + 1).astype(np.uint8)
    code |= np.where(np.signbit(p) & finite[:, None, :, None], 128, 0).astype(np.uint8)
    scales = np.where(finite, a / TOP, np.nan).astype(np.float32)
    return code.reshape(rows * block, cols * 128)[:R, :K].copy(), scales


def f8_values(codes, scales):
    """float64 values of a matrix [R, K]; the block follows from the scales' shape."""
    codes, scales = np.asarray(codes), np.asarray(scales, dtype=np.float64)
    R, K = codes.shape
    if scales.shape[0] != R or R == 1:
        scales = np.repeat(scales, 128, axis=0)[:R]
    return VALUES[codes] * np.repeat(scales, 128, axis=1)[:, :K]


def f8_gemm_ref(x, w, residual=None):
    """(y, the sum of the terms' magnitudes) of x . w^T + residual on float64 values."""
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    if residual is not None:
        y, a = y + residual, a + np.abs(residual)
    return y, a


def act_ref(g, act):
    """(act(g), act'(g))."""
    if act == "silu":
        e = np.exp(-np.abs(g))
        s = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s + g * e / (1 + e) ** 2
    c = np.sqrt(2 / np.pi)
    z = c * (g + 0.044715 * g ** 3)
    e = np.exp(-2 * np.abs(z))                        # 1 + tanh z = 2 s(2 z), tanh' = 4 e / (1 + e)^2
    s = np.where(z >= 0, 1 / (1 + e), e / (1 + e))
    return g * s, s + g * 2 * e / (1 + e) ** 2 * c * (1 + 3 * 0.044715 * g ** 2)


def gated_ref(x, w, act):
    """(h, g, u) of the float64 values x [M, K] and w [2F, K]."""
    p = x @ w.T
    F = w.shape[0] // 2
    g, u = p[:, :F], p[:, F:]
    return act_ref(g, act)[0] * u, g, u


def gated_grad_ref(dh, x, w, act):
    """The gradients [M, 2F] of the projections."""
    _, g, u = gated_ref(x, w, act)
    a, da = act_ref(g, act)
    return np.concatenate([dh * u * da, dh * a], axis=1)
