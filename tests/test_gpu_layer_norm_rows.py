"""layer_norm_rows, layer_norm_rows_backward and dropout_rows against the 64-bit oracle:
every way a row can lie on threads, odd widths, pitches, offsets of rows, empty and
single rows, infinities and NaN, dropped values, in-place calls, batch invariance,
64-bit places, guards, graphs and streams."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import training

from _layer import FLOOR, HALF, TYPES, U, f32, f64, ids, make, sum_depth
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def vector(rng, cols, dtype, mean=1.0, scale=0.3):
    return torch.from_numpy(mean + scale * rng.standard_normal(cols)).to(dtype).cuda()


def copy(t):
    """A copy whose rows start at multiples of 16 bytes."""
    m = torch.empty(t.shape[0], -(-t.shape[1] // 8) * 8, dtype=t.dtype, device=t.device)
    return m[:, :t.shape[1]].copy_(t)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def check_norm(r, h, w, b, eps):
    """out, mean and inv_std against the oracle on the sum h that was written."""
    cols, d = h.shape[1], sum_depth(h.shape[1])
    want, mean, inv = training.layer_norm(f64(h), f64(w), None if b is None else f64(b), eps)
    c = f64(h) - mean[:, None]
    dev, std = np.abs(c).mean(1), np.sqrt((c * c).mean(1))
    # A part's mean m is corrected by the sum of h - m: each difference and its additions
    # (d + 3) on the deviations, the corrected mean's own rounding and the joined one's on
    # the mean; parts of a row are joined from the first one's mean, which is at most 16
    # deviations off (16 parts), with at most 19 roundings on differences of means
    e_mean = U * (4 * np.abs(mean) + (d + 3 + 17 * 19) * dev)
    # squared deviations: two roundings, the additions, and for parts their means' errors
    # twice; where there are none, what the rounding of their cancellation leaves
    e_var = (d + 24) * U * std ** 2 + 4 * e_mean * std + \
        (d + 4) * U * ((d + 2) * U * np.abs(f64(h)).mean(1)) ** 2
    rel = (e_var / (2 * (std ** 2 + eps)) + 4 * U) * 1.02
    if r.mean is not None:
        assert np.all(np.abs(f64(r.mean) - mean) <= e_mean * 1.02)
        assert np.all(np.abs(f64(r.inv_std) - inv) <= rel * inv)
    aw, n = np.abs(f64(w)), np.abs(c) * inv[:, None]
    tol = (HALF[h.dtype] + U) * np.abs(want) + aw * (inv * e_mean)[:, None] + \
        aw * n * (rel[:, None] + 2 * U)
    bad = ~(np.abs(f64(r.out) - want) <= tol * 1.02 + FLOOR[h.dtype])
    assert not bad.any(), (np.argwhere(bad)[:4], f64(r.out)[bad][:4], want[bad][:4])


# every row_shape (8 .. 64 lanes; whole wavefronts with 1, 2 or 4 chunks a lane; the
# loop) at its ends, odd widths among them
COLS = [1, 2, 7, 8, 63, 64, 65, 128, 129, 250, 256, 257, 511, 512, 513, 1001, 1024, 1025, 2048,
        2049, 2056, 4096, 4097, 5001, 8192, 8193, 16384, 16391, 32768, 32769, 40000, 100003]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", COLS)
def test_norm_with_what_reaches_it(cols, dtype):
    rng = np.random.default_rng(cols)
    rows = 37 if cols <= 4096 else 5
    x = make(rng, rows, cols, dtype, 2.0, pad=1, device="cuda")
    res = make(rng, rows, cols, dtype, 1.0, pad=3, device="cuda")
    w, b = vector(rng, cols, dtype), vector(rng, cols, dtype, 0.0)
    plain = armx.layer_norm_rows(x, w, b, keep_stats=True)
    assert plain.sum is None
    check_norm(plain, x, w, b, 1e-5)
    r = armx.layer_norm_rows(x, w, residual=res, eps=1e-6, keep_stats=True)
    assert same(r.sum, (x.float() + res.float()).to(dtype))
    check_norm(r, r.sum, w, None, 1e-6)
    for residual in (res, None):
        drop = armx.Dropout(0.25, 11, 5)
        keep, scale = training.kept(0.25, 11, 5, rows, cols)
        want = training.dropout(f32(x), keep, scale, None if residual is None else f32(residual))
        r = armx.layer_norm_rows(x, w, b, residual=residual, dropout=drop, keep_stats=True)
        assert np.array_equal(f32(r.sum), f32(torch.from_numpy(want).to(dtype)))
        check_norm(r, r.sum, w, b, 1e-5)
        assert torch.equal(armx.dropout_rows(x, drop, residual=residual), r.sum)
        bare = armx.layer_norm_rows(x, w, b, residual=residual, dropout=drop)
        assert bare.mean is None and bare.inv_std is None and torch.equal(bare.out, r.out)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [8, 100, 1000, 5000, 16384, 40000])
def test_rows_far_from_zero_keep_their_variance(cols, dtype):
    # rows of m +- one or two steps of their type: sums of squares would lose the variance
    rng = np.random.default_rng(cols)
    rows = 6
    base = torch.tensor([0.0, 1.0, 64.0, -256.0, 1024.0, 128.0])[:, None]
    step = base.abs().clamp(min=1.0) * torch.finfo(dtype).eps
    x = make(rng, rows, cols, dtype, device="cuda")
    x.copy_(base + step * torch.from_numpy(rng.integers(0, 3, (rows, cols))))
    x[5] = 128.0   # a row of one value has no variance at all
    w, b = vector(rng, cols, dtype), vector(rng, cols, dtype, 0.0)
    for eps in (1e-5, 1e-12):
        check_norm(armx.layer_norm_rows(x, w, b, eps=eps, keep_stats=True), x, w, b, eps)


def check_backward(got, dy, h, w, mean, inv, ds, drop, place=None):
    rows, cols = h.shape
    d, dtype = sum_depth(cols), h.dtype
    dh, dw, db, (g, mg, mgn, n, i), sdw, sdb = training.layer_norm_backward(
        f64(dy), f64(h), f64(w), f64(mean), f64(inv), None if ds is None else f64(ds))
    # g, its difference from its mean, the next and inv's product one rounding each (5 with
    # the last on dh); the means the additions, their division and the same three; n two
    # roundings in the sum of g n and two where it is used
    tol = U * i * (5 * g + (d + 8) * mg + n * (d + 12) * mgn) + U * (0 if ds is None else np.abs(dh))
    def close(a, want, tol):
        bad = ~(np.abs(f64(a) - want) <= (HALF[dtype] * np.abs(want) + tol) * 1.02 + FLOOR[dtype])
        assert not bad.any(), (np.argwhere(bad)[:4], f64(a)[bad][:4], want[bad][:4])
    if drop is None:
        assert got.dresidual is None
        close(got.dx, dh, tol)
    else:
        keep, scale = training.kept(drop.p, drop.seed, place or drop.offset, rows, cols,
                                    drop.first_row)
        close(got.dresidual, dh, tol)
        close(got.dx, np.where(keep, dh * float(scale), 0.0),
              np.where(keep, (tol + U * np.abs(dh)) * float(scale), 0.0))
        assert not got.dx[torch.from_numpy(~keep).cuda()].any()
    # n two roundings, its product one, and no term meets more than rows + 8 additions
    assert np.all(np.abs(f64(got.dweight) - dw) <= (rows + 12) * U * 1.02 * sdw + 2.0 ** -149)
    assert np.all(np.abs(f64(got.dbias) - db) <= (rows + 9) * U * 1.02 * sdb + 2.0 ** -149)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [24, 100, 512, 1000, 4096, 5000, 16384, 40000])
def test_means_beside_large_deviations(cols, dtype):
    # values of one grid, whose every sum is exact in binary32, in pairs that cancel but for
    # one: what is left is the division, within a unit of the mean
    rng = np.random.default_rng(cols)
    a = rng.integers(-120, 121, (50, cols // 2))
    h = np.concatenate([a, -a, np.zeros((50, cols % 2), int)], 1)[:, rng.permutation(cols)]
    h[:, 3] = 0
    h[np.arange(50), 3] = np.arange(50) - 25 - (h.sum(1) - h[:, 3])
    x = torch.zeros(50, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]
    x.copy_(torch.from_numpy(h / 32.0))
    assert np.array_equal(f64(x), h / 32.0)
    w = torch.ones(cols, dtype=dtype, device="cuda")
    got = f64(armx.layer_norm_rows(x, w, keep_stats=True).mean)
    want = f64(x).sum(1) / cols
    assert np.all(np.abs(got - want) <= 2 * U * np.abs(want)), np.abs(got - want).max()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (2, 64), (3, 8), (1000, 64), (4099, 136),
                                       (513, 2056), (300, 8192), (70000, 16), (33, 33000),
                                       (512, 1001), (513, 1024), (1024, 2049), (1025, 4100),
                                       (1200, 7000), (300, 16384), (520, 16390), (90, 32768),
                                       (1100, 257), (5000, 33)])
@pytest.mark.parametrize("kind", ["alone", "dsum", "dropout", "both"])
def test_backward(rows, cols, dtype, kind):
    rng = np.random.default_rng(rows + cols)
    h = make(rng, rows, cols, dtype, 2.0, pad=2, device="cuda")
    dy = make(rng, rows, cols, dtype, 0.5, pad=1, device="cuda")
    ds = make(rng, rows, cols, dtype, 0.25, device="cuda") if kind in ("dsum", "both") else None
    drop = armx.Dropout(0.1, 3 << 40, 9) if kind in ("dropout", "both") else None
    w = vector(rng, cols, dtype)
    s = armx.layer_norm_rows(h, w, keep_stats=True)
    got = armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std, dsum=ds, dropout=drop)
    check_backward(got, dy, h, w, s.mean, s.inv_std, ds, drop)


def test_backward_against_differences_of_the_forward():
    rng = np.random.default_rng(5)
    # whole steps that are exact in 16 bits
    h = torch.from_numpy(rng.integers(-64, 65, (6, 40)) / 16).half().cuda()
    w = torch.from_numpy(rng.integers(8, 25, 40) / 16).half().cuda()
    dy = torch.from_numpy(rng.integers(-16, 17, (6, 40)) / 16).half().cuda()
    s = armx.layer_norm_rows(h, w, keep_stats=True)
    dx = f64(armx.layer_norm_rows_backward(dy, h, w, s.mean, s.inv_std).dx)
    step = 1 / 16
    for j in (0, 3, 17, 39):
        e = torch.zeros_like(h)
        e[:, j] = step
        ends = [h + e, h - e]
        got = [f64(armx.layer_norm_rows(v, w).out) for v in ends]
        want = [training.layer_norm(f64(v), f64(w), None, 1e-5)[0] for v in ends]
        diff, exact = (((a - b) * f64(dy)).sum(1) / (2 * step) for a, b in (got, want))
        # the forward's results are half a step of theirs off (and their statistics a
        # thousandth of that); the quotient's own curvature is taken from 64 bits
        off = ((np.abs(want[0]) + np.abs(want[1])) * HALF[torch.float16] * 1.01
               * np.abs(f64(dy))).sum(1) / (2 * step)
        assert np.all(np.abs(diff - exact) <= off + 1e-6)
        deriv = training.layer_norm_backward(f64(dy), f64(h), f64(w), f64(s.mean), f64(s.inv_std))[0]
        assert np.all(np.abs(diff - dx[:, j]) <= off + np.abs(exact - deriv[:, j])
                      + HALF[torch.float16] * 1.05 * np.abs(dx[:, j]) + 1e-5)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (1000, 24), (257, 100), (64, 512),
                                       (33, 1001), (9, 4104), (3, 20000), (2, 40001), (0, 64),
                                       (5, 0)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(rows, cols, dtype, p):
    rng = np.random.default_rng(rows + cols)
    x, r = (make(rng, rows, cols, dtype, pad=i, device="cuda") for i in (1, 2))
    step = torch.tensor([(1 << 33) + 5], device="cuda")
    drop = armx.Dropout(p, (1 << 64) - 3, (1 << 35) + 1, step=step, first_row=12345)
    keep, scale = training.kept(p, drop.seed, drop.offset + int(step), rows, cols, 12345)
    for residual in (None, r):
        got = armx.dropout_rows(x, drop, residual=residual)
        want = training.dropout(f32(x), keep, scale, None if residual is None else f32(residual))
        assert np.array_equal(f32(got), f32(torch.from_numpy(want).to(dtype)))
    out = copy(x)
    assert armx.dropout_rows(out, drop, out=out) is out
    assert np.array_equal(f32(out), f32(armx.dropout_rows(x, drop)))
    out = copy(r)
    armx.dropout_rows(x, drop, residual=out, out=out)
    assert torch.equal(out, got)


def test_dropout_drops_whatever_stood_there():
    x = torch.full((4, 4096), float("nan"), dtype=torch.float16, device="cuda")
    x[1], x[2] = float("inf"), -float("inf")
    drop = armx.Dropout(0.5, 77)
    keep = torch.from_numpy(training.kept(0.5, 77, 0, 4, 4096)[0]).cuda()
    y = armx.dropout_rows(x, drop)
    assert not y[~keep].any() and torch.equal(y[1][keep[1]], x[1][keep[1]])
    assert torch.isnan(y[0][keep[0]]).all()
    assert not armx.dropout_rows(x, armx.Dropout(1.0, 77)).any()
    r = torch.ones_like(x)
    assert torch.equal(armx.dropout_rows(x, armx.Dropout(1.0, 77), residual=r), r)
    # through the norm a dropped NaN is as if it were not there, forward and back
    x[3] = torch.randn(4096).half()
    x[3][~keep[3]] = float("nan")
    w = torch.ones(4096, dtype=torch.float16, device="cuda")
    n = armx.layer_norm_rows(x, w, residual=r, dropout=drop, keep_stats=True)
    assert torch.isfinite(n.out[3]).all() and torch.isnan(n.out[:3]).any(1).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [24, 300, 5000, 40000])
def test_what_is_not_finite_stays_in_its_row(cols, dtype):
    rng = np.random.default_rng(cols)
    x = make(rng, 6, cols, dtype, device="cuda")
    x[1, cols // 2], x[3, 0], x[4, -1] = float("nan"), float("inf"), -float("inf")
    w = vector(rng, cols, dtype)
    n = armx.layer_norm_rows(x, w, keep_stats=True)
    assert torch.isnan(n.out[[1, 3, 4]]).all()
    fine = [0, 2, 5]
    check_norm(armx.LayerNorm(n.out[fine], None, n.mean[fine], n.inv_std[fine]), x[fine], w, None, 1e-5)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(40, 200), (5, 4100), (700, 1000), (1500, 1000), (3, 40000)])
def test_in_place(rows, cols, dtype):
    rng = np.random.default_rng(rows)
    x, r, dy = (make(rng, rows, cols, dtype, device="cuda") for _ in range(3))
    w, b = vector(rng, cols, dtype), vector(rng, cols, dtype, 0.0)
    drop = armx.Dropout(0.1, 4)
    want = armx.layer_norm_rows(x, w, b, residual=r, dropout=drop, keep_stats=True)
    for o, s in ((0, 1), (1, 0)):
        pair = [copy(x), copy(r)]
        got = armx.layer_norm_rows(pair[0], w, b, residual=pair[1], dropout=drop, out=pair[o],
                                   sum_out=pair[s], keep_stats=True)
        assert got.out is pair[o] and torch.equal(pair[o], want.out)
        assert torch.equal(pair[s], want.sum) and torch.equal(got.mean, want.mean)
    grads = armx.layer_norm_rows_backward(dy, want.sum, w, want.mean, want.inv_std, dsum=r,
                                          dropout=drop)
    for o, s in ((0, 1), (1, 0)):
        pair = [copy(dy), copy(r)]
        got = armx.layer_norm_rows_backward(pair[0], want.sum, w, want.mean, want.inv_std,
                                            dsum=pair[1], dropout=drop, out=pair[o], dresidual=pair[s])
        assert torch.equal(pair[o], grads.dx) and torch.equal(pair[s], grads.dresidual)
        assert torch.equal(got.dweight, grads.dweight) and torch.equal(got.dbias, grads.dbias)
    h = copy(want.sum)   # dy, dsum and h one tensor
    one = armx.layer_norm_rows_backward(h, h, w, want.mean, want.inv_std, dsum=h)
    got = armx.layer_norm_rows_backward(h, h, w, want.mean, want.inv_std, dsum=h, out=h)
    assert all(torch.equal(a, c) for a, c in zip(got[:3], one[:3]))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [64, 100, 1000, 4096, 9000, 40000])
def test_a_row_does_not_depend_on_the_others(cols, dtype):
    rng = np.random.default_rng(cols)
    rows = 70
    x, r, dy = (make(rng, rows, cols, dtype, device="cuda") for _ in range(3))
    w, b = vector(rng, cols, dtype), vector(rng, cols, dtype, 0.0)
    d = armx.Dropout(0.2, 6, first_row=(1 << 32) - rows)
    all_ = armx.layer_norm_rows(x, w, b, residual=r, dropout=d, keep_stats=True)
    g = armx.layer_norm_rows_backward(dy, all_.sum, w, all_.mean, all_.inv_std, dsum=r, dropout=d)
    for at, n in ((0, 1), (69, 1), (13, 20)):
        part = slice(at, at + n)
        dp = d._replace(first_row=d.first_row + at)
        one = armx.layer_norm_rows(x[part], w, b, residual=r[part], dropout=dp, keep_stats=True)
        assert all(torch.equal(a, c[part]) for a, c in zip(one, all_))
        gp = armx.layer_norm_rows_backward(dy[part], one.sum, w, one.mean, one.inv_std,
                                           dsum=r[part], dropout=dp)
        assert torch.equal(gp.dx, g.dx[part]) and torch.equal(gp.dresidual, g.dresidual[part])


def test_no_rows_and_no_columns():
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    n = armx.layer_norm_rows(x, w, w, residual=x, dropout=armx.Dropout(0.1, 1), keep_stats=True)
    assert n.out.shape == (0, 64) and n.mean.shape == (0,)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    g = armx.layer_norm_rows_backward(x, x, w, n.mean, n.inv_std, dweight=dw, dbias=db)
    assert g.dx.shape == (0, 64) and not dw.any() and not db.any()
    x = torch.empty(5, 0, dtype=torch.float16, device="cuda")
    n = armx.layer_norm_rows(x, w[:0], keep_stats=True)
    assert not n.mean.any() and not n.inv_std.any()


def test_places_past_32_bits():
    rows, cols = 70000, 32768   # 2^31 values and more
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    d = armx.Dropout(0.1, 5)
    y = armx.layer_norm_rows(x, w, dropout=d)
    for at in (0, 65535, 65536, rows - 1):
        one = armx.layer_norm_rows(x[at:at + 1], w, dropout=d._replace(first_row=at))
        assert torch.equal(one.out[0], y.out[at]) and torch.equal(one.sum[0], y.sum[at])
    check_norm(armx.LayerNorm(y.out[-2:], None, None, None), y.sum[-2:], w, None, 1e-5)


def test_results_stay_inside_their_rows():
    rng = np.random.default_rng(1)
    for rows, cols in ((5, 13), (300, 100), (1500, 1001), (3, 40001)):
        mark = 123.0
        outs = [torch.full((rows + 2, -(-cols // 8) * 8 + 8), mark, dtype=torch.bfloat16, device="cuda")
                for _ in range(4)]
        views = [o[1:-1, :cols] for o in outs]
        x, r, dy = (make(rng, rows, cols, torch.bfloat16, device="cuda") for _ in range(3))
        w = vector(rng, cols, torch.bfloat16)
        sums = torch.full((2, cols + 8), mark, device="cuda")
        d = armx.Dropout(0.1, 2)
        n = armx.layer_norm_rows(x, w, residual=r, dropout=d, keep_stats=True, out=views[0],
                                 sum_out=views[1])
        armx.layer_norm_rows_backward(dy, n.sum, w, n.mean, n.inv_std, dropout=d, out=views[2],
                                      dresidual=views[3], dweight=sums[0, 4:4 + cols],
                                      dbias=sums[1, 4:4 + cols])
        armx.dropout_rows(x, d, out=views[1])
        for o, v in zip(outs, views):
            assert torch.isfinite(v).all()
            v.fill_(mark)
            assert (o == mark).all()
        assert (sums[:, :4] == mark).all() and (sums[:, 4 + cols:] == mark).all()


def test_refused_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    w, d = x[0], armx.Dropout(0.1, 1)
    stat = torch.zeros(4, device="cuda")
    for call, error, match in [
            (lambda: armx.dropout_rows(x, None), TypeError, "must be a Dropout"),
            (lambda: armx.dropout_rows(x, (0.1, 1)), TypeError, "must be a Dropout"),
            (lambda: armx.dropout_rows(x, d._replace(p=1.5)), ValueError, "from 0 to 1"),
            (lambda: armx.dropout_rows(x, d._replace(p=float("nan"))), ValueError, "from 0 to 1"),
            (lambda: armx.dropout_rows(x, d._replace(seed=-1)), ValueError, "2\\^64"),
            (lambda: armx.dropout_rows(x, d._replace(seed=1 << 64)), ValueError, "2\\^64"),
            (lambda: armx.dropout_rows(x, d._replace(offset=1.0)), TypeError, "must be an int"),
            (lambda: armx.dropout_rows(x, d._replace(step=torch.zeros(1, dtype=torch.long))),
             ValueError, "step must be 1"),
            (lambda: armx.dropout_rows(x, d._replace(step=stat[:1])), ValueError, "step must be 1"),
            (lambda: armx.dropout_rows(x, d._replace(first_row=1 << 32)), armx.ArmxError, "SHAPE"),
            (lambda: armx.layer_norm_rows(x, w[:63]), ValueError, "weight"),
            (lambda: armx.layer_norm_rows(x, w, w.bfloat16()), ValueError, "bias"),
            (lambda: armx.layer_norm_rows(x, w, sum_out=x), ValueError, "sum_out goes with"),
            (lambda: armx.layer_norm_rows(x, w, residual=x[:3]), ValueError, "residual"),
            (lambda: armx.layer_norm_rows(x, w, eps=-1.0), armx.ArmxError, "CONFIG"),
            (lambda: armx.layer_norm_rows(x.t(), w[:4]), ValueError, "contiguous"),
            (lambda: armx.layer_norm_rows_backward(x, x, w, stat, stat, dresidual=x), ValueError,
             "dresidual goes with"),
            (lambda: armx.layer_norm_rows_backward(x, x, w, stat[:3], stat), ValueError, "mean"),
            (lambda: armx.layer_norm_rows_backward(x, x, w, stat, stat, dropout=d, out=x, dresidual=x),
             armx.ArmxError, "CONFIG")]:
        with pytest.raises(error, match=match):
            call()


def test_results_given_count_as_written():
    x = torch.ones(4, 64, dtype=torch.float16, device="cuda")
    w, d, stat = x[0].clone(), armx.Dropout(0.1, 1), torch.ones(4, device="cuda")
    o, s, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda"), \
        torch.empty(64, device="cuda")
    for call, written in [
            (lambda: armx.dropout_rows(x, d, out=o), (o,)),
            (lambda: armx.layer_norm_rows(x, w, residual=x, out=o, sum_out=s), (o, s)),
            (lambda: armx.layer_norm_rows_backward(x, x, w, stat, stat, dropout=d, out=o, dresidual=s,
                                                   dweight=dw, dbias=db), (o, s, dw, db))]:
        before = [t._version for t in (x, w, stat, *written)]
        call()
        after = [t._version for t in (x, w, stat, *written)]
        assert after[:3] == before[:3] and all(a > b for a, b in zip(after[3:], before[3:]))
