"""The scale that binary16's values of dz have for dx: no value leaves binary16's range,
and the target's own is a power of two, whatever the sizes of the logits, how sure the row
is, and how far its log of the sum of exponentials is off within the roundings that it may
have."""
import numpy as np
import pytest

from oracle import training
from oracle.binary16 import decode_table
from oracle.mfma_model import GROUP, group_step

LARGEST = 65504.0
U = 2.0 ** -24


def scaled(z, size, lse):
    """dz of the two words of rows, the target first, times the rows' scales."""
    z, lse = z.astype(np.float32), np.asarray(lse, np.float32)[:, None]
    with np.errstate(over="ignore"):
        dz = np.exp(z - lse, dtype=np.float32)
    dz[:, 0] -= np.float32(1)
    return dz * training.row_scale(z[:, 0], size, lse[:, 0])[:, None], dz


@pytest.mark.parametrize("off", [-8, -1, 0, 1, 8])
def test_range_at_any_logit(off):
    # off: roundings of the summed magnitudes that lse is off by
    rng = np.random.default_rng(off + 9)
    n = 200000
    size = np.float32(2.0 ** rng.uniform(-2, 20, n))
    hit = np.float32(size * rng.uniform(-1, 1, n) ** 3)   # cancelling, mostly
    rest = 2.0 ** rng.uniform(-24, -0.01, n)              # true 1 - p, all of it one word's
    lse = hit - np.log1p(-rest)
    z = np.stack((hit, np.float32(lse + np.log(rest))), 1)
    got, dz = scaled(z, size, lse + off * U * size)
    assert np.abs(got).max() <= LARGEST
    least = 2.0 ** 14 / training.row_scale(hit, size, hit)
    clear = np.abs(dz[:, 0]) >= least
    assert np.allclose(np.abs(got[clear, 0]), 2.0 ** 14, rtol=4 * U, atol=0) and clear.sum() > n / 4
    # no scale is larger than a row that is only a little sure of its target needs
    assert np.all(least <= np.maximum(2.0 ** -14, size * 2.0 ** -20) * (1 + 4 * U))


def chain(x, w):
    """The matrix units' sum of products in the reconstructed order, a binary32."""
    q, _ = decode_table()
    p = [int(a) * int(b) for a, b in zip(q[x.view(np.uint16)], q[w.view(np.uint16)])]
    acc = 0
    for i in range(0, len(p), GROUP):
        acc = group_step(acc, p[i:i + GROUP])
    return np.ldexp(float(acc), -48)


@pytest.mark.parametrize("cols", [1024, 4096, 8192])
@pytest.mark.parametrize("logit", [40, 400, 2000])
def test_range_with_the_matrix_units_sums(logit, cols):
    rng = np.random.default_rng(logit + cols)
    rows = 16384 // cols * 3
    x = rng.standard_normal((rows, cols))
    along = x / (x * x).sum(1, keepdims=True)
    noise = rng.standard_normal((rows, cols)) * logit / (6.25 * cols ** 0.5)
    noise -= (noise * x).sum(1, keepdims=True) * along
    rest = 10.0 ** rng.uniform(-5, -2, rows)
    w = noise + logit * along
    words = [w, w + np.log(rest / (1 - rest))[:, None] * along]
    xh = x.astype(np.float16)
    z = np.array([[chain(xh[r], v[r].astype(np.float16)) for v in words] for r in range(rows)])
    size = np.abs(xh.astype(float) * w.astype(np.float16)).sum(1)
    got, _ = scaled(z, size, np.float32(np.logaddexp(z[:, 0], z[:, 1])))
    assert np.abs(got).max() <= LARGEST
