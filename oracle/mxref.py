"""Plain NumPy oracle of the MXFP4 operators (microscaled 4-bit floating point:
E2M1 elements in blocks of 32 with one E8M0 scale), in 64 bits and without the
library's code.

Codes are uint8 [R, K/2], element 2i of a row in the low nibble of byte i;
scales are uint8 [R, K/32], the byte s standing for 2^(s - 127), 255 for NaN."""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize(x):
    """(codes, scales) of x [R, K] by the definition: the scale's exponent is
    floor(log2 of the block's largest magnitude) - 2, at least -127; an element
    goes to the nearest value, of two equally near to the one with the even
    code.  A block with an infinity or NaN has the scale 255 and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    b = np.where(finite[:, :, None], b, 0.0)
    _, ex = np.frexp(np.abs(b).max(axis=2))           # magnitude = m 2^ex, m in [0.5, 1)
    e = np.where((b != 0).any(axis=2), np.maximum(ex - 1 - 2, -127), -127)
    m = np.ldexp(np.abs(b), -e[:, :, None])
    gap = np.abs(m[..., None] - VALUES)
    best = gap.min(axis=-1, keepdims=True)
    near = gap == best                               # one value, or two at the same distance
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1)).astype(np.uint8)
    code |= np.where(np.signbit(b), 8, 0).astype(np.uint8)
    code = np.where(finite[:, :, None], code, 0).reshape(R, K).astype(np.uint8)
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scales


def mx_values(codes, scales):
    """float64 values of an MXFP4 matrix [..., K]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    n = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(n >= 8, -VALUES[n & 7], VALUES[n & 7])
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def mx_gemm_ref(x, w, residual=None):
    """(y, the sum of the terms' magnitudes) of x . w^T + residual on float64 values."""
    y, a = x @ w.T, np.abs(x) @ np.abs(w).T
    if residual is not None:
        y, a = y + residual, a + np.abs(residual)
    return y, a


def mx_grouped_ref(x, w, offsets, rows=None, row_scale=None, fill=0.0):
    """As mx_gemm_ref for groups: w [E, N, K]; rows outside the groups hold `fill`."""
    T = len(rows) if rows is not None else x.shape[0]
    y = np.full((T, w.shape[1]), float(fill))
    a = np.zeros((T, w.shape[1]))
    for e in range(w.shape[0]):
        for t in range(offsets[e], offsets[e + 1]):
            r = t if rows is None else rows[t]
            if r < 0 or r >= x.shape[0]:
                y[t] = 0.0
                continue
            f = 1.0 if row_scale is None else float(row_scale[t])
            y[t] = (w[e] @ x[r]) * f
            a[t] = (np.abs(w[e]) @ np.abs(x[r])) * abs(f)
    return y, a
