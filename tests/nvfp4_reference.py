"""The NVFP4 code of fp32 values as include/dvl.h defines a cache's, every fp32
operation rounded once (NumPy)."""
from __future__ import annotations

import numpy as np

from cache_reference import E4M3

F = np.float32
_POSITIVE = E4M3[:0x7f]
_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def nearest_even(x, values):
    """Index of the nearest of rising values (the nearest of even index between
    two), the last one for larger x."""
    x = np.asarray(x, dtype=np.float64)
    i = np.clip(np.searchsorted(values, x, side="right") - 1, 0, len(values) - 2)
    low, high = x - values[i], values[i + 1] - x
    return np.where(x >= values[-1], len(values) - 1, np.where((low < high) | ((low == high) & (i % 2 == 0)), i, i + 1))


def encode(y, scale):
    """y [.., D] -> (codes [.., D/2], block scales [.., D/16]), both uint8."""
    y = np.asarray(y, dtype=F).reshape(*np.shape(y)[:-1], -1, 16)
    s = nearest_even(np.abs(y).max(axis=-1) / F(F(6) * F(scale)), _POSITIVE).astype(np.uint8)
    unit = (E4M3[s].astype(F) * F(scale))[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s[..., None] == 0, F(0), y / unit)
    assert z.dtype == F
    c = nearest_even(np.abs(z), _E2M1) + 8 * np.signbit(z)
    c = c.reshape(*y.shape[:-2], -1, 2).astype(np.uint8)
    return c[..., 0] | c[..., 1] << 4, s


def ties(rng, rows, heads, D, scale):
    """bf16 values of which many quotients lie in the middle between two codes:
    a block's largest value sets its scale s, the others are s scale times the
    middles (where those are bf16 numbers) or anything."""
    middles = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    # block scales of three bits whose products with the middles fit bf16's eight
    s = E4M3[rng.integers(0x20, 0x60, size=(rows, heads, D // 16, 1))]
    y = s * middles[rng.integers(7, size=(rows, heads, D // 16, 16))]
    y[..., rng.integers(16)] = 6 * s[..., 0]
    y = np.where(rng.random(y.shape) < 0.1, y * rng.random(y.shape), y) * rng.choice([-1, 1], size=y.shape)
    return (y * scale).reshape(rows, heads, D)
