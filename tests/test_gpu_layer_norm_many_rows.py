"""layer_norm_rows, layer_norm_rows_backward and dropout_rows on many rows, where other
kernels run than on few: blocks that walk over rows, gradients from blocks' partial sums
(two chunks a thread among them), results written past the caches; against 64 bits, in every
way that a row of up to 16384 values lies on threads, with NaN behind the rows."""
from functools import lru_cache

import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import training

from _layer import FLOOR, HALF, TYPES, U, ids, sum_depth
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# 2^24 values and more, which are written past the caches
PAST = [(270000, 63), (135000, 128), (70000, 250), (34000, 500), (17000, 1001), (12000, 1500),
        (8200, 2056), (4200, 4096), (4150, 4101), (2060, 8192), (2060, 8193), (1030, 16384)]
# and fewer, with partial sums of two chunks a thread, and others
FEWER = [(1100, 2056), (1500, 3001), (1030, 4096), (2100, 4088), (1100, 1030)]


def normal(gen, rows, cols, dtype, scale=1.0, pad=1):
    m = torch.full((rows, (-(-cols // 8) + pad) * 8), float("nan"), dtype=dtype,
                   device="cuda")[:, :cols]
    return m.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)


def vector(gen, cols, dtype, mean=1.0):
    return (mean + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)


@lru_cache(maxsize=2)
def kept(rows, cols):
    keep, scale = training.kept(0.25, 7 << 33, 21, rows, cols)
    return torch.from_numpy(keep).cuda(), float(scale)


DROP = armx.Dropout(0.25, 7 << 33, 21)


def sums_depth(rows, cols):
    """No term of dweight or dbias meets more than this many additions: a thread's rows,
    those that its block takes at a time, the join's 32 threads and what each of them adds."""
    p = armx.launch_plan(armx.OP_LAYER_NORM_BACKWARD, rows, cols)
    assert p["launches"] == 2, p
    per = 32 if cols <= 64 else 16 if cols <= 128 else 8 if cols <= 256 else 4 if cols <= 512 else 1
    return -(-(-(-rows // per)) // p["grid_blocks"]) + per + -(-p["grid_blocks"] // 32) + 32


def inside(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    at = tuple(bad.nonzero()[0].tolist()) if bad.any() else None
    assert at is None, (int(bad.sum()), at, float(got[at]), float(want[at]))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("kind", ["plain", "residual", "dropout", "both"])
@pytest.mark.parametrize("rows,cols", PAST)
def test_norm(rows, cols, kind, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = normal(gen, rows, cols, dtype, 2.0)
    res = normal(gen, rows, cols, dtype, 1.0, 2) if kind in ("residual", "both") else None
    drop = DROP if kind in ("dropout", "both") else None
    w, b = vector(gen, cols, dtype), vector(gen, cols, dtype, 0.0)
    r = armx.layer_norm_rows(x, w, b, residual=res, dropout=drop, keep_stats=True)
    h = x
    if kind != "plain":
        want = x.float()
        if drop:
            keep, scale = kept(rows, cols)
            want = torch.where(keep, want * scale, 0.0)
            alone = armx.dropout_rows(x, drop, residual=res)
        if res is not None:
            want = want + res.float()
        h = r.sum
        assert torch.equal(h, want.to(dtype)) and (not drop or torch.equal(alone, h))
        del want
    else:
        assert r.sum is None
    # mean and deviations as test_gpu_layer_norm_rows.py has them
    H, W = h.double(), w.double()
    mean = H.mean(1)
    c = H - mean[:, None]
    dev, std, d = c.abs().mean(1), (c * c).mean(1).sqrt(), sum_depth(cols)
    inv = ((c * c).mean(1) + 1e-5).rsqrt()
    e_mean = U * (4 * mean.abs() + (d + 3 + 17 * 19) * dev)
    e_var = (d + 24) * U * std ** 2 + 4 * e_mean * std
    rel = (e_var / (2 * (std ** 2 + 1e-5)) + 4 * U) * 1.02
    inside(r.mean, mean, e_mean * 1.02)
    inside(r.inv_std, inv, rel * inv)
    n = c * inv[:, None]
    want = n * W + b.double()
    tol = (HALF[dtype] + U) * want.abs() + W.abs() * ((inv * e_mean)[:, None]
                                                    + n.abs() * (rel[:, None] + 2 * U))
    inside(r.out, want, tol * 1.02 + FLOOR[dtype])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("kind", ["alone", "dsum", "dropout", "both"])
@pytest.mark.parametrize("rows,cols", PAST + FEWER)
def test_backward(rows, cols, kind, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    h = normal(gen, rows, cols, dtype, 2.0)
    dy = normal(gen, rows, cols, dtype, 0.5, 2)
    ds = normal(gen, rows, cols, dtype, 0.25, 0) if kind in ("dsum", "both") else None
    drop = DROP if kind in ("dropout", "both") else None
    w = vector(gen, cols, dtype)
    s = armx.layer_norm_rows(h, w, keep_stats=True)
    got = armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std, dsum=ds, dropout=drop)
    Y, i, d = dy.double(), s.inv_std.double()[:, None], sum_depth(cols)
    n, g = (h.double() - s.mean.double()[:, None]) * i, Y * w.double()
    dh = i * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    # as test_gpu_layer_norm_rows.py has them
    tol = U * i * (5 * g.abs() + (d + 8) * g.abs().mean(1, keepdim=True)
                   + n.abs() * (d + 12) * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dh = dh + ds.double()
        tol = tol + U * dh.abs()
    half, floor = HALF[dtype], FLOOR[dtype]
    if drop is None:
        assert got.dresidual is None
        inside(got.dx, dh, (half * dh.abs() + tol) * 1.02 + floor)
    else:
        keep, scale = kept(rows, cols)
        inside(got.dresidual, dh, (half * dh.abs() + tol) * 1.02 + floor)
        want, tol = dh * keep * scale, (tol + U * dh.abs()) * scale
        inside(got.dx, want, (half * want.abs() + tol) * 1.02 + floor)
        assert not got.dx[~keep].any()
    depth = sums_depth(rows, cols)
    inside(got.dweight, (Y * n).sum(0), (depth + 3) * U * 1.02 * (Y * n).abs().sum(0) + 2.0 ** -149)
    inside(got.dbias, Y.sum(0), depth * U * 1.02 * Y.abs().sum(0) + 2.0 ** -149)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1030, 4096), (4200, 4096), (34000, 500)])
def test_gradients_in_place_and_again(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    h, dy, ds = (normal(gen, rows, cols, dtype, k, p) for k, p in ((2.0, 1), (0.5, 2), (0.25, 0)))
    w = vector(gen, cols, dtype)
    s = armx.layer_norm_rows(h, w, keep_stats=True)
    want = armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std, dsum=ds, dropout=DROP)
    again = armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std, dsum=ds, dropout=DROP)
    got = armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std, dsum=ds, dropout=DROP, out=dy,
                                        dresidual=ds)
    assert got.dx is dy and got.dresidual is ds
    for other in (again, got):
        assert all(torch.equal(a, b) for a, b in zip(other, want))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", PAST + [(600, 32768), (430, 40001)])
def test_dropout(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, res = normal(gen, rows, cols, dtype), normal(gen, rows, cols, dtype, 1.0, 2)
    keep, scale = kept(rows, cols)
    want = torch.where(keep, x.float() * scale, 0.0)
    assert torch.equal(armx.dropout_rows(x, DROP), want.to(dtype))
    assert torch.equal(armx.dropout_rows(x, DROP, residual=res), (want + res.float()).to(dtype))
