"""Plain 64-bit forms (NumPy) of what goes into a paged cache and what comes out
of a 4-bit one, written from the definitions in include/dvl.h, with the error
bounds the tests use.  u is half an fp32 ulp, relative (2^-24)."""
from __future__ import annotations

import numpy as np

from step_reference import BF16, U, e4m3_values

E4M3 = e4m3_values()
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def decode(codes, blocks, scale):
    """Codes [..][D/2] (low nibble = even d) and E4M3 codes of the scales [..][D/16] -> values [..][D]."""
    x = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], axis=-1).reshape(*codes.shape[:-1], -1, 16)
    return (x * E4M3[blocks][..., None] * scale).reshape(*codes.shape[:-1], -1)


def turned(x, weight, eps, positions, freqs, interleaved):
    """Norm and rotation of x [rows][heads][D].  Returns (values, error bound).

    The mean of D squares carries at most D / 8 + 8 roundings (a lane's chain of
    eight, a butterfly of five, the division), half of them reach its root, the
    reciprocal root a few more; weights, cos, sin and the two products one each:
    48 u covers D = 256.  cos and sin are off by at most 2^-20 (2^-21.2 of the
    fast units, 2^-22 of an angle within half a turn rounded to fp32)."""
    D = x.shape[-1]
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * weight
    size = np.abs(y)
    out = y.copy()
    if freqs is not None:
        half = len(freqs)
        first = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
        second = first + (1 if interleaved else half)
        t = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freqs)
        a, b = y[..., first], y[..., second]
        out[..., first] = a * np.cos(t) - b * np.sin(t)
        out[..., second] = b * np.cos(t) + a * np.sin(t)
        size = size.copy()
        size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
        return out, size * (2.0 ** -20 + 48 * U) + 1e-37
    assert D <= 256
    return out, size * 48 * U + 1e-37


def bf16_bound(z, err):
    return BF16 * (np.abs(z) + err) + err


def check_e4m3(codes, z, err, scale):
    """Codes against RNE_e4m3(z / scale): half a step (2^-4 relative, 2^-10 below
    the normal numbers) of a quotient off by err / scale and two roundings."""
    want = np.clip(z / scale, -448, 448)
    slack = err / scale + 4 * U * np.abs(want)
    off = np.abs(E4M3[codes] - want)
    tol = 2.0 ** -4 * (np.abs(want) + slack) + 2.0 ** -10 + slack
    assert np.all(off <= tol), (off - tol).max()


def check_nvfp4(codes, blocks, z, err, scale):
    """Codes and scales against the definition: the scale within half an E4M3
    step of max |z| / (6 scale), and with the scale that was stored every value
    within half an E2M1 step of z (or saturated, or all zero)."""
    rows = z.reshape(*z.shape[:-1], -1, 16)
    e = err.reshape(rows.shape)
    big = np.abs(rows).max(axis=-1)
    want = np.minimum(big / (6 * scale), 448)
    s = E4M3[blocks]
    slack = e.max(axis=-1) / (6 * scale) + 6 * U * want
    assert np.all(np.abs(s - want) <= 2.0 ** -4 * (want + slack) + 2.0 ** -10 + slack)
    x = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], axis=-1).reshape(rows.shape)
    unit = (s * scale)[..., None]
    step = np.where(np.abs(x) < 2, 0.25, np.where(np.abs(x) < 4, 0.5, 1.0))
    # the lower neighbour's step counts at 2 and 4, where the steps change, only
    # downwards; the larger is allowed for both
    over = np.maximum(np.abs(rows) - 6 * unit, 0)
    tol = np.where(unit > 0, step * unit + over, np.abs(rows)) + e + 6 * U * np.abs(rows)
    off = np.abs(x * unit - rows)
    assert np.all(off <= tol), (off - tol).max()
    assert np.all(x[s == 0] == 0)


def places(rows, lengths, starts=None):
    """[(sequence, place)] of each row, (-1, 0) past the last sequence."""
    B = len(lengths)
    starts = [rows // B * b for b in range(B + 1)] if starts is None else list(starts)
    out = [(-1, 0)] * rows
    for b in range(B):
        for r in range(starts[b], starts[b + 1]):
            out[r] = (b, int(lengths[b]) - (starts[b + 1] - r))
    return out


def kept(pool, table, lengths, first, keep, counts):
    """pool [pages][page][..] after the kept tokens moved."""
    pages, page = pool.shape[:2]
    out = pool.copy()
    for b in range(len(lengths)):
        limit = min(int(lengths[b]), table.shape[1] * page)
        f = max(int(first[b]), 0)
        for i in range(max(0, min(int(counts[b]), keep.shape[1]))):
            src, dst = f + int(keep[b, i]), f + i
            if keep[b, i] < 0 or src >= limit or dst >= limit:
                continue
            p, q = int(table[b, src // page]), int(table[b, dst // page])
            if 0 <= p < pages and 0 <= q < pages:
                out[q, dst % page] = pool[p, src % page]
    return out
