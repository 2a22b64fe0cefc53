"""cross_entropy_rows_backward on rows that are nearly sure of their target: large logits
whose sums cancel, where 1 - p is close to what the logits' own rounding leaves, and
probabilities beside a large log of the sum of exponentials."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx

from _layer import FLOOR, HALF, TYPES, U, f64, ids
from _parity import require_gpu
from test_gpu_cross_entropy import check_grads, check_loss

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


def nearly_sure(rng, cols, logit, dtype, rows=120, most=-2):
    """Row r's target is word 2 r, and word 2 r + 1 is the only other one near it: half the
    rows have 1 - p from 1e-5 to 10^most, the others from 2.4e-4 to 4e-4.  What the words
    have beside the row's own direction cancels in its logits, and is many times them."""
    x = rng.standard_normal((rows, cols))
    along = x / (x * x).sum(1, keepdims=True)
    noise = rng.standard_normal((rows, cols)) * logit / (6.25 * cols ** 0.5)
    noise -= (noise * x).sum(1, keepdims=True) * along
    rest = np.where(np.arange(rows) % 2, 10.0 ** rng.uniform(-5, most, rows),
                    rng.uniform(2.4e-4, 4e-4, rows))
    w = np.empty((2 * rows, cols))
    w[::2] = noise + logit * along
    w[1::2] = w[::2] + np.log(rest / (1 - rest))[:, None] * along
    return put(x, dtype), put(w, dtype), torch.arange(0, 2 * rows, 2, device="cuda")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [1001, 4096, 8192])
@pytest.mark.parametrize("logit", [100, 400, 1000, 4000])
def test_large_logits_of_rows_nearly_sure(logit, cols, dtype):
    rng = np.random.default_rng(logit + cols)
    x, w, t = nearly_sure(rng, cols, logit, dtype)
    rows, vocab = x.shape[0], w.shape[0]
    got = armx.cross_entropy_rows(x, w, t)
    check_loss(got, x, w, t)
    # (a loss scale of 1024, so that binary16's results keep their bits)
    dloss = torch.from_numpy(rng.uniform(512, 1536, rows).astype(np.float32)).cuda()
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse, dweight_dtype=torch.float32)
    assert torch.isfinite(g.dx).all() and torch.isfinite(g.dweight).all()
    check_grads(g, dloss, x, w, t, got.lse)
    # Both gradients are made of the same dz, which dweight (two terms up to 128 rows)
    # shows: word v's row of it is dz[r][v] x[r] of its one row r, as every other word is
    # 0.3 logits and more behind.  dx has a rounding of each of its two dz, floors at the
    # smallest step of what is scaled to 2^14 over at most 1, and its own rounding.
    xs, ws, dw = f64(x), f64(w), f64(g.dweight)
    half, floor, ag = HALF[dtype], FLOOR[dtype], f64(dloss)[:, None]
    mine = np.repeat(xs, 2, 0)
    dz = ((dw * mine).sum(1) / (mine * mine).sum(1)).reshape(rows, 2)
    want = dz[:, :1] * ws[::2] + dz[:, 1:] * ws[1::2]
    size = np.abs(dz[:, :1] * ws[::2]) + np.abs(dz[:, 1:] * ws[1::2])
    floors = floor * ag.max() * (2.0 ** -14 + 2.0 ** -15)
    far = ag * vocab * np.exp(-0.2 * logit)
    tol = size * (half + half ** 2 + (2 * (vocab + 40) + 30) * U) + (floors + far) * (
        np.abs(ws).sum(0) + np.abs(ws).max())
    bad = ~(np.abs(f64(g.dx) - want) <= (tol + half * (np.abs(want) + tol)) * 1.02 + floor)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], f64(g.dx)[bad][:4], want[bad][:4])


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


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows", [100, 128, 129, 4096])
def test_a_word_of_one_token(rows, dtype):
    # Its row of dweight is one value of dz times that token's x, and no other rounding
    # averages with its own: half a step of the 16-bit type on either side of 128 rows, and
    # up to them two terms' square of it.
    rng = np.random.default_rng(rows)
    vocab, cols, token = 500, 64, rows // 3
    x = rng.integers(-3, 4, (rows, cols)) / 4   # logits that are exact
    w = rng.integers(-1, 2, (vocab, cols)) / 4
    x[:, 0] = 3
    x[token, 0] = -0.75
    w[vocab - 1] = 0
    w[vocab - 1, 0] = -8        # 24 behind for the others, 6 before for its token
    t = rng.integers(0, vocab - 1, rows)
    t[token] = vocab - 1
    xd, wd, td = put(x, dtype), put(w, dtype), torch.from_numpy(t).cuda()
    lse = armx.cross_entropy_rows(xd, wd, td).lse
    dloss = torch.from_numpy(rng.uniform(0.5, 1.5, rows).astype(np.float32)).cuda()
    g = armx.cross_entropy_rows_backward(dloss, xd, wd, td, lse, dweight_dtype=torch.float32)
    d = x @ w[vocab - 1] - f64(lse)
    p = np.exp(d)
    dz = (p - (np.arange(rows) == token)) * f64(dloss)
    assert np.abs(np.delete(dz, token)).max() < 1e-6 * abs(dz[token])
    want = dz @ x
    e_p = (p * U * (3 * np.abs(d) + 4)) * f64(dloss) + FLOOR[dtype] * 1.5 * 2.0 ** -15
    size = np.abs(dz) @ np.abs(x)
    rest = e_p @ np.abs(x) + (2 * (2 * rows + 40) + 4) * U * size
    err = np.abs(f64(g.dweight)[vocab - 1] - want)
    assert np.all(err <= (HALF[dtype] * size + rest) * 1.02)
    if rows <= 128:
        assert np.all(err <= (HALF[dtype] ** 2 * size + rest) * 1.02)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [600, 1001, 4096])
@pytest.mark.parametrize("logit", [100, 400])
def test_a_target_s_value_is_exact_in_dx(logit, cols, dtype):
    # A column that no logit sees and in which targets' words have 1: dx there is dz of the
    # row's target, which is a power of two in 16 bits if its scale is made of the same
    # logit, bit for bit: it has dx's own rounding and no other.  dweight, where x is 1, has
    # that dz in two terms.
    rng = np.random.default_rng(logit * cols)
    x, w, t = nearly_sure(rng, cols, logit, dtype, most=-0.5)
    x[:, 0], x[:, 1], w[:, 0] = 0, 1, 0
    w[::2, 0] = 1
    rows = x.shape[0]
    z = f64(x) @ f64(w).T
    far = np.arange(2 * rows) // 2 != np.arange(rows)[:, None]
    assert (z - np.diag(z[:, ::2])[:, None])[far].max() < -20   # no other row's words
    lse = armx.cross_entropy_rows(x, w, t).lse
    dloss = torch.from_numpy(rng.uniform(512, 1536, rows).astype(np.float32)).cuda()
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, lse, dweight_dtype=torch.float32)
    dz, got, half = f64(g.dweight)[::2, 1], f64(g.dx)[:, 0], HALF[dtype]
    # rows no surer than the magnitudes that are summed allow
    size = (np.abs(f64(x)) * np.abs(f64(w)[::2])).sum(1)
    clear = np.abs(dz) > 1.01 * f64(dloss) * np.maximum(2.0 ** -14, 2.0 ** -20 * size)
    assert clear.sum() > 10
    tol = np.abs(dz) * (half * (1 + half) + half ** 2 + 16 * U) + FLOOR[dtype] * 1536 * 2.0 ** -14
    assert np.all((np.abs(got - dz) <= tol + FLOOR[dtype])[clear]), \
        (np.abs(got - dz) / np.abs(dz) / half)[clear].max()
