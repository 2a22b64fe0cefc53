"""Every tile in every product of the cross entropy and its gradients, with one step of 64
values and several, cut and whole, against 64 bits; and a row's bits in every tile.

SHAPES names the tiles that a shape takes on 256 compute units, of the logits, of dx (with
the parts that its sum is cut into) and of dweight; test_tile16_choice.py checks the names.
The logits' tile is the loss's too where the vocabulary is one piece, as it is here."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx

from _layer import FLOOR, HALF, TYPES, U, ids
from _parity import require_gpu

pytestmark = pytest.mark.gpu

SHAPES = {
    # logits 256 x 256 of 3 and 4 steps and more
    (200, 50001, 135): "256x256 128x128/64 256x256",
    (200, 50001, 192): "256x256 64x128/32 256x256",
    (200, 50001, 197): "256x256 64x128/32 256x256",
    (200, 50001, 256): "256x256 64x128/32 256x256",
    (700, 20000, 200): "256x256 128x128/16 256x128",
    (1000, 16384, 2051): "256x256 192x256/4 256x128",
    (3000, 16384, 1000): "256x256 192x256/4 256x256",
    (3000, 16384, 2056): "256x256 256x256/2 256x128",
    # dx 256 x 256, 192 x 256 and 256 x 128 of 1 to 5 steps
    (6000, 20, 2056): "16x64 256x256/1 16x64",
    (6000, 64, 2051): "16x64 256x256/1 16x64",
    (6000, 100, 2056): "16x64 256x256/1 16x64",
    (6000, 128, 2051): "16x64 256x256/1 16x64",
    (6000, 150, 2056): "64x128 256x256/1 16x64",
    (6000, 192, 2056): "64x128 256x256/1 16x64",
    (6000, 200, 2056): "64x128 256x256/1 16x64",
    (6000, 256, 2056): "64x128 256x256/1 16x64",
    (6000, 300, 2051): "128x128 256x256/1 16x64",
    (4096, 20, 2056): "16x64 192x256/1 16x64",
    (4096, 64, 2051): "16x64 192x256/1 16x64",
    (4096, 150, 2056): "16x64 192x256/1 16x64",
    (4096, 192, 2051): "16x64 192x256/1 16x64",
    (4096, 300, 2056): "64x128 192x256/1 16x64",
    (2048, 20, 2051): "16x64 256x128/1 16x64",
    (2048, 128, 2056): "16x64 256x128/1 16x64",
    (2048, 150, 2051): "16x64 256x128/1 16x64",
    (2048, 300, 2056): "16x64 256x128/1 16x64",
    (6000, 100, 135): "16x64 64x128/1 16x64",
    (8192, 100, 72): "16x128 16x128/1 16x64",
    # dweight 256 x 256 and 192 x 256 of 1 to 5 steps; other tiles of the logits
    (70, 50001, 136): "128x128 64x128/64 256x256",
    (96, 50001, 135): "128x128 64x128/64 256x256",
    (128, 50001, 136): "128x128 64x128/64 256x256",
    (257, 50001, 136): "192x256 256x128/64 256x256",
    (1, 40000, 136): "16x64 16x64/64 192x256",
    (32, 40000, 135): "64x128 16x64/64 192x256",
    (33, 40000, 136): "64x128 16x64/64 192x256",
    (64, 40000, 136): "64x128 16x64/64 192x256",
    (100, 40000, 135): "128x128 64x128/64 192x256",
    (129, 40000, 256): "192x256 64x128/32 192x256",
    (257, 40000, 136): "128x128 256x128/64 192x256",
    # and the others
    (129, 50001, 8): "192x256 16x64/64 128x128",
    (129, 50001, 72): "192x256 64x128/64 128x128",
    (100, 40000, 8): "128x128 16x64/64 256x128",
    (257, 40000, 7): "128x128 128x128/64 256x128",
    (1, 50001, 8): "16x128 16x64/64 128x128",
    (777, 5000, 200): "256x128 64x128/8 64x128",
    (200, 20000, 200): "256x128 64x128/32 256x128",
    (515, 20000, 8): "192x256 128x128/32 128x128",
    (1, 8192, 72): "16x64 16x64/16 16x128",
    (777, 5000, 8): "128x128 16x64/8 16x64",
}

# (rows, the tile of their loss) against 20000 words of 200 values
BATCHES = [(1, "16x64"), (16, "16x64"), (33, "16x128"), (65, "128x128"), (129, "64x128"),
           (200, "256x128"), (400, "192x256"), (700, "256x256")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def put(values, dtype):
    """On the GPU, rows at multiples of 16 bytes, NaN behind them."""
    rows, cols = values.shape
    m = torch.full((rows, (cols + 15) // 8 * 8), float("nan"), dtype=dtype, device="cuda")[:, :cols]
    m.copy_(torch.from_numpy(values))
    return m


def exact_inputs(rng, rows, vocab, cols, dtype):
    """Quarters, whose products' sums are exact in binary32; logits of a deviation of about
    4, so that few words have most of a row's probability."""
    x = rng.integers(-3, 4, (rows, cols)) / 4
    w = rng.integers(-1, 2, (vocab, cols)) * (max(1, round(4 / (0.41 * cols ** 0.5))) / 4)
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < 0.2] = -100
    if rows > 1:
        t[rows - 1] = vocab - 1
    return put(x, dtype), put(w, dtype), torch.from_numpy(t).cuda()


def off(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[:4].tolist()
        return int(bad.sum()), at, [float(got[tuple(i)]) for i in at], [float(want[tuple(i)]) for i in at]
    return None


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,vocab,cols", SHAPES)
def test_every_tile(rows, vocab, cols, dtype):
    rng = np.random.default_rng(rows + vocab + cols)
    x, w, t = exact_inputs(rng, rows, vocab, cols, dtype)
    X, W, live = x.double(), w.double(), t != -100
    z = X @ W.t().contiguous()
    lse = torch.logsumexp(z, 1)
    got = armx.cross_entropy_rows(x, w, t)
    # An exponential: the difference, its product with log2 e and that constant, each a
    # rounding of an exponent of at most the row's span, and the instruction's unit, then
    # alike the factors of the joined sums; 6 additions of 64, 8 + 16 and one per 128 pieces;
    # the logarithm good to 2 units, its sum with the largest logit one.
    span = z.amax(1) - z.amin(1)
    e_lse = U * (2 * (3 * span + 4) + 30 + vocab / 8192 + 4 * np.log(vocab) + 4 + 2 * lse.abs())
    assert off(got.lse, lse, e_lse * 1.02) is None
    hit = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(live, lse - hit, 0.0)
    assert off(got.loss, loss, (e_lse + U * loss.abs()) * 1.02) is None
    assert not got.loss[~live].any()

    dloss = torch.from_numpy(rng.uniform(0.5, 1.5, rows).astype(np.float32)).cuda()
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse)
    wide = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse, dweight_dtype=torch.float32)
    assert torch.equal(wide.dx, g.dx)
    # dz's exponentials as above, of the given lse, and one addition
    d = z - got.lse.double()[:, None]
    p = torch.exp(d)
    e_p = p * (U * (3 * d.abs() + 4))
    del z, d
    p[live, t[live]] -= 1.0
    ag = torch.where(live, dloss.double(), 0.0)[:, None]
    dz, half, floor = p * ag, HALF[dtype], FLOOR[dtype]
    adz = dz.abs()
    # a rounding of dz to 16 bits behind two products, floors at binary16's smallest step
    # (2^14 stands for 1 - p of the target, 2^15 for the largest |dloss|), the sums' additions
    e = e_p * ag
    e_dz = adz * (half + 3 * U) + e + floor * ag * 2.0 ** -13
    tol = e_dz @ W.abs() + 2 * U * (vocab + 40) * (adz @ W.abs())
    want = dz @ W
    assert off(g.dx, want, (tol + half * (want.abs() + tol)) * 1.02 + floor) is None
    assert not g.dx[~live].any()
    once = half if rows > 128 else half ** 2
    e_dz = (adz * (once + 4 * U) + e + floor * float(ag.max()) * 2.0 ** -15).t().contiguous()
    tol = e_dz @ X.abs() + 2 * U * (2 * rows + 40) * (adz.t().contiguous() @ X.abs())
    want = dz.t().contiguous() @ X
    assert off(wide.dweight, want, (tol + U * (want.abs() + tol)) * 1.02 + 2.0 ** -149) is None
    assert off(g.dweight, want, (tol + half * (want.abs() + tol)) * 1.02 + floor) is None


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_a_row_has_the_same_bits_in_every_tile(dtype):
    rng = np.random.default_rng(5)
    vocab, cols = 20000, 200
    x = put(rng.standard_normal((900, cols)), dtype)
    w = put(rng.standard_normal((vocab, cols)) * 0.2, dtype)
    t = torch.from_numpy(rng.integers(0, vocab, 900)).cuda()
    want = armx.cross_entropy_rows(x, w, t)
    for n, _ in BATCHES:
        got = armx.cross_entropy_rows(x[99:99 + n], w, t[99:99 + n])
        assert torch.equal(got.loss, want.loss[99:99 + n]), n
        assert torch.equal(got.lse, want.lse[99:99 + n]), n


@pytest.mark.parametrize("rows,vocab,cols,dtype", [(515, 32003, 1000, torch.float16),
                                                   (3000, 16384, 1000, torch.bfloat16),
                                                   (100, 50001, 136, torch.bfloat16)])
def test_calls_repeat_themselves(rows, vocab, cols, dtype):
    # bits depend on nothing but the inputs; the last calls' workspaces hold other calls'
    rng = np.random.default_rng(rows)
    x = put(rng.standard_normal((rows, cols)), dtype)
    w = put(rng.standard_normal((vocab, cols)) * cols ** -0.5, dtype)
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    dloss = torch.rand(rows, device="cuda")
    want = armx.cross_entropy_rows(x, w, t)
    grads = armx.cross_entropy_rows_backward(dloss, x, w, t, want.lse)
    for _ in range(5):
        other = armx.cross_entropy_rows(x[: rows // 2], w, t[: rows // 2])
        armx.cross_entropy_rows_backward(dloss[: rows // 2], x[: rows // 2], w, t[: rows // 2],
                                         other.lse, dweight_dtype=torch.float32)
        got = armx.cross_entropy_rows(x, w, t)
        assert torch.equal(got.loss, want.loss) and torch.equal(got.lse, want.lse)
        again = armx.cross_entropy_rows_backward(dloss, x, w, t, want.lse)
        assert torch.equal(again.dx, grads.dx) and torch.equal(again.dweight, grads.dweight)
