"""fp64 restatement of rotary positions, the 8-bit cache's rounding and the attention of one
token (test infrastructure: plain numpy, from the formulas of include/usp.h)."""
from __future__ import annotations

import numpy as np


def rope(x, positions, freqs, axes=None, interleaved=False, back=False):
    """x [tokens][H][D] turned by positions [n_axes][tokens]; (result, |x1| + |x2| of each element's pair)."""
    x = np.asarray(x, np.float64)
    n = len(freqs)
    axes = np.zeros(n, int) if axes is None else np.asarray(axes)
    w = np.asarray(positions, np.float64)[axes].T * np.asarray(freqs, np.float64)   # [tokens][pairs]
    c, s = np.cos(w)[:, None], np.sin(w)[:, None] * (-1.0 if back else 1.0)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y, size = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def to_e4m3(x):
    """(e4m3 values, exponents) of rows x [..., D]: the smallest e >= -126 with |x| <= 448 2^e in the whole row
    (infinities as the largest finite bf16, NaN aside), x / 2^e to the nearest value, ties to even, at most 448."""
    x = np.asarray(x, np.float64)
    most = float(2 ** 127 * (2 - 2.0 ** -7))
    size = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), most).max(-1)
    e = np.full(size.shape, -126)
    while True:
        low = size > 448.0 * np.exp2(e.astype(np.float64))
        if not low.any():
            break
        e = e + low
    with np.errstate(invalid="ignore"):
        y = x / np.exp2(e.astype(np.float64))[..., None]
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -200))), -6.0) - 3.0)
        y = np.where(np.isfinite(y), np.round(y / np.where(np.isfinite(step), step, 1.0)) * step, y)
    return np.clip(y, -448.0, 448.0), e


def decode(q, k, v, scale, sink=None):
    """One query q [D] over k, v [n][D] -> (O, LSE, sum p |v|, largest sum |q_d k_d| scale)."""
    s = (k @ q) * scale
    z = np.concatenate([s, [] if sink is None else [sink]])
    if z.size == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    m = z.max()
    lse = m + np.log(np.exp(z - m).sum())
    p = np.exp(s - lse)
    return p @ v, lse, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale) if len(s) else 0.0
