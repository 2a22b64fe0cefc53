"""cross_entropy_rows_backward on rows that are nearly sure of their target: probabilities
beside a large log of the sum of exponentials."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx

from _layer import FLOOR, HALF, TYPES, U, f64, ids
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def put(values, dtype):
    """On the GPU, rows at multiples of 16 bytes."""
    rows, cols = values.shape
    m = torch.empty(rows, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]
    m.copy_(torch.from_numpy(values))
    return m


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_probabilities_beside_a_large_lse(dtype):
    # Logits that are exact, and an lse that is what it is in binary32: the exponent z - lse
    # is exact where 1 - p is small, so p has the instruction's unit (U below 1) and the
    # exponent's product with log2 e, three roundings of a number about 1 - p.
    # Rows have columns of their own, so every logit but a row's target's is 0.
    rng = np.random.default_rng(12)
    rows, cols = 64, 512
    x, w = np.zeros((rows, cols)), np.zeros((2 * rows, cols))
    for r in range(rows):
        x[r, 8 * r:8 * r + 8] = rng.integers(4, 13, 8) * rng.choice([-1, 1], 8)
        w[r, 8 * r:8 * r + 8] = np.sign(x[r, 8 * r:8 * r + 8]) * rng.integers(8, 129) / 4
    hit = (x * w[:rows]).sum(1)
    assert hit.min() > 50 and hit.max() > 1000
    lse = (hit + 10.0 ** rng.uniform(-5, -1.5, rows)).astype(np.float32)
    rest = -np.expm1(hit - lse)
    assert (rest > 0).sum() > rows / 2
    dloss = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    xd, wd, t = put(x, dtype), put(w, dtype), torch.arange(rows, device="cuda")
    g = armx.cross_entropy_rows_backward(torch.from_numpy(dloss).cuda(), xd, wd, t,
                                         torch.from_numpy(lse).cuda(),
                                         dweight_dtype=torch.float32)
    half, floor = HALF[dtype], FLOOR[dtype]
    e_dz = dloss * (1.5 * U + 4 * U * rest)
    want = -(rest * dloss)[:, None] * x
    off = np.abs(f64(g.dweight)[:rows] - want)
    # two terms, a factor back and the one product's additions; the last term's floor
    tol = (e_dz + rest * dloss * (half ** 2 + 20 * U) + floor * 1.5 * 2.0 ** -15)[:, None] * np.abs(x)
    assert np.all(off <= tol * 1.02 + 1e-15), off.max()
    # dx: a rounding of dz besides, and of the result
    want = -(rest * dloss)[:, None] * w[:rows]
    tol = (e_dz + rest * dloss * (half + 20 * U) + floor * 1.5 * 2.0 ** -14)[:, None] * np.abs(w[:rows])
    tol = tol + 1e-14 * np.abs(w).sum(0)
    off = np.abs(f64(g.dx) - want)
    assert np.all(off <= (tol + half * (np.abs(want) + tol)) * 1.02 + floor)
