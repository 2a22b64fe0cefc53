"""Layer norm, dropout and the cross entropy of rows from their definitions, in
binary64 (numpy), for the tests.  Inputs are float32 or float64 arrays holding values
of a 16-bit type."""
from __future__ import annotations

import numpy as np

LOW = np.uint64(0xFFFFFFFF)
HIGH = np.uint64(32)


def philox(counter, key):
    """Philox4x32-10 of four counter words (arrays that broadcast) and two key words."""
    x = [np.asarray(c, np.uint64) & LOW for c in counter]
    k = [int(v) & 0xFFFFFFFF for v in key]
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> HIGH) ^ x[1] ^ np.uint64(k[0]), b & LOW,
             (a >> HIGH) ^ x[3] ^ np.uint64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def kept(p, seed, offset, rows, cols, first_row=0):
    """Which values a dropout keeps, and the binary32 that they are multiplied by."""
    limit = int(65536 * p + 0.5)
    place = offset % 2 ** 64
    words = philox((np.arange(-(-cols // 8))[None, :], np.arange(first_row, first_row + rows)[:, None],
                    place & 0xFFFFFFFF, place >> 32), (seed, seed >> 32))
    words = np.stack(np.broadcast_arrays(*words), 2)
    bits = np.stack((words & np.uint64(0xFFFF), words >> np.uint64(16)), 3).reshape(rows, 8 * -(-cols // 8))[:, :cols]
    return bits >= limit, np.float32(65536 / (65536 - limit) if limit < 65536 else 0)


def dropout(x, keep, scale, residual=None):
    """Binary32 result before it is rounded to 16 bits: each step one rounding."""
    y = np.where(keep, np.asarray(x, np.float32) * scale, np.float32(0))
    return y if residual is None else y + np.asarray(residual, np.float32)


def layer_norm(h, w, b, eps):
    """(norm, mean, 1 / standard deviation) of the rows of h, unrounded."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    mean = h.mean(1)
    d = h - mean[:, None]
    inv = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * inv[:, None] * w + (0.0 if b is None else np.asarray(b, np.float64)), mean, inv


def layer_norm_backward(dy, h, w, mean, inv, dsum=None):
    """(dh, dweight, dbias), unrounded, with what bounds their roundings: |g|, the means
    of |g| and of |g n|, |n| and inv, for dh, and the sums of |dy n| and |dy| over rows."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    mean, inv = np.asarray(mean, np.float64)[:, None], np.asarray(inv, np.float64)[:, None]
    n, g = (h - mean) * inv, dy * w
    dh = inv * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    if dsum is not None:
        dh = dh + np.asarray(dsum, np.float64)
    bounds = (np.abs(g), np.abs(g).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True),
              np.abs(n), inv)
    return dh, (dy * n).sum(0), dy.sum(0), bounds, np.abs(dy * n).sum(0), np.abs(dy).sum(0)


def cross_entropy(x, w, targets, ignore=-100):
    """(loss, lse, z) of the rows of x against the rows of w."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    t = np.asarray(targets)
    inside = (t >= 0) & (t < z.shape[1])
    hit = z[np.arange(len(t)), np.where(inside, t, 0)]
    return np.where(t == ignore, 0.0, np.where(inside, lse - hit, np.nan)), lse, z


def cross_entropy_backward(dloss, x, w, targets, lse, ignore=-100):
    """(dx, dweight, dz), unrounded, for targets inside the vocabulary or ignored, whose
    rows of x reach nothing."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    t = np.asarray(targets)
    live = t != ignore
    x = np.where(live[:, None], x, 0.0)
    dz = np.exp(x @ w.T - np.asarray(lse, np.float64)[:, None])
    rows = np.flatnonzero(live)
    dz[rows, t[rows]] -= 1.0
    dz = np.where(live[:, None], dz * np.where(live, dloss, 0.0)[:, None], 0.0)
    return dz @ w, dz.T @ x, dz


def row_scale(z, size, lse):
    """What a row of exp(z - lse) - onehot(target) is multiplied by before binary16 holds
    it, in binary32: z and lse as the kernel has them, size = sum |x w| of the target's
    logit."""
    z, size, lse = (np.float32(v) for v in (z, size, lse))
    least = np.minimum(np.maximum(size * np.float32(2.0 ** -20), np.float32(2.0 ** -14)), np.float32(1))
    rest = np.maximum(np.abs(np.float32(1) - np.exp(z - lse, dtype=np.float32)), least)
    return np.float32(2.0 ** 14) / rest
