"""Norms of rows, 8-bit codes and products of codes from their definitions, in
binary64 (numpy), for the tests.  Inputs are float32 or float64 arrays holding
values of a 16-bit type."""
from __future__ import annotations

import numpy as np


def rms_norm(h, w, eps):
    """(norm, 1 / rms) of the rows of h, unrounded."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    inv = 1.0 / np.sqrt((h * h).sum(1) / h.shape[1] + eps)
    return h * inv[:, None] * w, inv


def rms_norm_backward(dy, h, w, inv, dsum=None):
    """(dx, dweight), unrounded, and the sums of magnitudes behind each:
    |g| inv, |h| inv^3 mean |g h|, and sum over rows of |dy h inv|."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    inv = np.asarray(inv, np.float64)[:, None]
    g = dy * w
    dx = inv * (g - h * inv ** 2 * (g * h).mean(1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    n = dy * h * inv
    return (dx, n.sum(0), np.abs(g) * inv,
            np.abs(h) * inv ** 3 * np.abs(g * h).mean(1, keepdims=True), np.abs(n).sum(0))


def codes(p):
    """Codes and largest magnitudes of the rows of p (binary32 values): round
    half to even of the exact 127 p / max|p|.  Zeros for a row of zeros; zeros
    and NaN for a row that is not finite."""
    p = np.asarray(p, np.float64)
    top = np.abs(p).max(1, initial=0.0, keepdims=True)
    fine = np.isfinite(p).all(1, keepdims=True)
    a = np.where(fine, np.abs(p), 0.0)
    t = np.where(fine & (top > 0), top, 1.0)
    # numerator and denominator scaled by powers of two into whole numbers of
    # at most 24 and 32 bits apart in binary64: every product below is exact
    e = np.exp2(-np.floor(np.log2(t)))
    a, t = a * e, t * e
    k = np.floor(127 * a / t)
    k = np.where(2 * k * t > 254 * a, k - 1, k)
    k = np.where(2 * (k + 1) * t <= 254 * a, k + 1, k)
    twice, border = 254 * a, (2 * k + 1) * t
    k = k + ((twice > border) | ((twice == border) & (k % 2 == 1)))
    q = np.where(p < 0, -k, k)
    return (np.where(fine, q, 0).astype(np.int8), np.where(fine, top, np.nan)[:, 0])


def product(a, b):
    """Exact integer sums of products of the rows of a and b."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return a @ b.T   # below 2^53: exact
