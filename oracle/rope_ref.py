"""Float64 reference of the rotary positions, written from the definition (include/diffattn.h): every part of
d channels of a row turned pair by pair, and rounding to bf16 in one step. Test infrastructure: the library
never calls it."""
from __future__ import annotations

import numpy as np


def table(inv_freq, top: int):
    """cos and sin [top, pairs, 2] in float64."""
    a = np.arange(top, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    return np.stack([np.cos(a), np.sin(a)], -1)


def pair_channels(i: int, pairs: int, interleaved: bool):
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def rotate(x, tab, positions, d: int, axes=None, interleaved=False, inverse=False):
    """Rows x [total, heads, width] turned; tab [top, pairs, 2], positions [total] or [n, total]. Rows of tokens
    left out (a position of -1) come back as they are."""
    y = np.array(x, dtype=np.float64)
    tab, pos = np.asarray(tab, dtype=np.float64), np.atleast_2d(np.asarray(positions))
    pairs = tab.shape[1]
    live = np.all(pos >= 0, axis=0)
    for i in range(pairs):
        p = np.where(live, pos[0 if axes is None else int(axes[i])], 0)
        c, s = tab[p, i, 0][:, None], tab[p, i, 1][:, None] * (-1.0 if inverse else 1.0)
        lo, hi = pair_channels(i, pairs, interleaved)
        for first in range(0, y.shape[2], d):
            x1, x2 = y[:, :, first + lo].copy(), y[:, :, first + hi].copy()
            y[:, :, first + lo] = np.where(live[:, None], x1 * c - x2 * s, x1)
            y[:, :, first + hi] = np.where(live[:, None], x2 * c + x1 * s, x2)
    return y


def to_bf16(x):
    """x in float64 rounded to bf16's 8 bits (ties to even) in one step, as float64; subnormals in steps of 2^-133."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
    with np.errstate(invalid="ignore"):
        y = np.round(x / step) * step
    y = np.where(np.isfinite(x), y, x)
    return np.where(np.abs(y) > 3.3895313892515355e38, np.copysign(np.inf, y), y)
