"""Plain 64-bit forms of the drafting step's operators (NumPy), written from
their definitions in include/dvl.h, and the error bounds the tests use.

u is half an fp32 ulp, relative (2^-24).  Rounding to bf16 moves a value by
at most 2^-8 of it (8 significant bits: half an ulp of 2^(e-7) against a
value of at least 2^e is 2^-8)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
BF16 = 2.0 ** -8


def e4m3_values() -> np.ndarray:
    """The value of each E4M3 code: 4 exponent bits (bias 7), 3 mantissa bits,
    no infinities, 0x7f and 0xff NaN."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7f) == 0x7f else (f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
        out[c] = -v if c & 0x80 else v
    return out


def norm(x, weight, residual, eps):
    """(u, y) in 64 bits."""
    u = x.astype(np.float64) + (0 if residual is None else residual.astype(np.float64))
    y = u / np.sqrt((u * u).mean(axis=1, keepdims=True) + eps) * weight.astype(np.float64)
    return u, y


def group_amax(y, group):
    K = y.shape[1]
    size = group or K
    return np.stack([np.abs(y[:, i:i + size]).max(axis=1) for i in range(0, K, size)], axis=1)


def attention(q, k, v, table, lengths, scale):
    """q [B][T][Hq][D], k and v [pages][page][heads][D] (values, scales applied).
    Returns (out, lse, tolerance of out, tolerance of lse) with the weights
    rounded by `w` relative, filled in by the caller through the returned
    pieces: out, lse, A = sum p |v|, S = largest bound of a score's error,
    V1 = sum |v|."""
    B, T, Hq, D = q.shape
    page, heads = k.shape[1], k.shape[2]
    G = Hq // heads
    out = np.zeros((B, T, Hq, D))
    A = np.zeros((B, T, Hq, D))
    V1 = np.zeros((B, T, Hq, D))
    S = np.zeros((B, T, Hq))
    lse = np.full((B, T, Hq), -np.inf)
    for b in range(B):
        length = max(0, min(int(lengths[b]), table.shape[1] * page))
        ids = table[b, :-(-length // page)]
        kk = k[ids].reshape(-1, heads, D)[:length]
        vv = v[ids].reshape(-1, heads, D)[:length]
        for t in range(T):
            n = length - (T - 1 - t)
            if n <= 0:
                continue
            for h in range(Hq):
                kh, vh = kk[:n, h // G], vv[:n, h // G]
                s = scale * (kh @ q[b, t, h])
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[b, t, h] = p @ vh
                A[b, t, h] = p @ np.abs(vh)
                V1[b, t, h] = np.abs(vh).sum(axis=0)
                lse[b, t, h] = m + np.log(e.sum())
                # D products summed in fp32 in any order, one scaling
                S[b, t, h] = abs(scale) * (np.abs(kh) @ np.abs(q[b, t, h])).max() * (D + 4) * U
    return out, lse, A, S, V1


def attention_bounds(out, lse, A, S, V1, n_max, fp8):
    """Tolerances of (out, lse).  Scores are off by at most S; a weight's
    exponent also carries the rounding of the score in log2 units (|s| u a few
    times, inside S's D + 4) and ex2's 2^-22; the weight is rounded to bf16
    (2^-8) or f16 (2^-11, and 2^-25 absolute below its normal range, with the
    sum of weights at least 1); the sums of n weights add n / 16 u (four
    weights per thread and tile, then the join)."""
    w = 2.0 ** -11 if fp8 else BF16
    rel = w + 2 * (S + 2.0 ** -21)[..., None] + (n_max / 16 + 64) * U
    tol = BF16 * np.abs(out) + rel * A * (1 + BF16) + (2.0 ** -24 * V1 if fp8 else 0) + 1e-30
    finite = np.isfinite(lse)
    tol_lse = np.where(finite, S + 2.0 ** -20 + (n_max / 16 + 64) * U + 8 * U * np.abs(np.where(finite, lse, 0)), 0)
    return tol, tol_lse


def beam_scores(logits, scores):
    """score(j, n) in 64 bits, [batch][beams][N]; NaN becomes -inf (no candidate)."""
    x = logits.astype(np.float64)
    with np.errstate(all="ignore"):
        m = x.max(axis=2, keepdims=True)
        lse = m + np.log(np.exp(x - m).sum(axis=2, keepdims=True))
        s = scores.astype(np.float64)[:, :, None] + (x - lse)
    return np.where(np.isnan(s), -np.inf, s)


def beam_tolerance(logits, scores):
    """A score's error: the subtraction and the addition round once each, lse
    once more and its sum by at most ~100 u (32 per thread, three butterflies,
    the chunks) plus the exponentials' few ulps."""
    fin = np.where(np.isfinite(logits), np.abs(logits.astype(np.float64)), 0).max()
    sc = np.where(np.isfinite(scores), np.abs(scores.astype(np.float64)), 0).max()
    return 4 * U * (2 * fin + sc + 25) + 200 * U
