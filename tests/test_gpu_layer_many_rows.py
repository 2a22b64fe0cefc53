"""The layer operators on many rows, where other kernels run than on few: blocks that walk
over rows, results written past the caches, dweight from blocks' partial sums; at odd widths
and narrow ones, with NaN behind the rows."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _layer import FLOOR, HALF, TYPES, U, f32, f64, ids, sum_depth
from _parity import require_gpu
from test_gpu_layer_norm import bits, check_codes, check_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def pitched(rows, cols, dtype, pad=1, fill=float("nan")):
    pitch = (-(-cols // 8) + pad) * 8
    return torch.full((rows, pitch), fill, dtype=dtype, device="cuda")[:, :cols]


def normal(gen, rows, cols, dtype, scale=1.0, pad=1):
    m = pitched(rows, cols, dtype, pad)
    m.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)
    return m


def whole(gen, rows, cols, dtype, top, pad=1):
    """Whole numbers of -top .. top."""
    m = pitched(rows, cols, dtype, pad)
    m.copy_(torch.randint(-top, top + 1, (rows, cols), generator=gen, device="cuda",
                          dtype=torch.int8))
    return m


def weight(gen, cols, dtype):
    return (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)


def rows_per_block(cols):
    """Rows that a block of the backward pass takes at a time."""
    return 32 if cols <= 64 else 16 if cols <= 128 else 8 if cols <= 256 else 4 if cols <= 512 else 1


def dweight_depth(rows, cols):
    """No term of dweight meets more than this many binary32 additions (the first, to
    zero, among them)."""
    p = armx.launch_plan(armx.OP_RMS_BACKWARD, rows, cols)
    if p["launches"] == 1:
        # a thread of a column block adds every block_threads / lanes-th row (lanes: 4 or 8,
        # the more the deeper), then 4 across lanes and its block's wavefronts
        return -(-rows // (p["block_threads"] // 8)) + 4 + p["block_threads"] // 64
    per = rows_per_block(cols)
    rounds = -(-(-(-rows // per)) // p["grid_blocks"])
    return rounds + per + -(-p["grid_blocks"] // 32) + 32


SPOTS = [0, 1, 2, 0.25, 0.5, 0.7, -3, -2, -1]


def spots(rows):
    """Rows to look at one by one: the ends and some between."""
    return sorted({int(s * rows) if isinstance(s, float) else s % rows for s in SPOTS})


# odd widths on every layout of a row, more than 1024 rows of each; the last three more
# than 2^24 values
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("rows,cols", [(5000, 37), (2111, 61), (40000, 101), (1031, 251),
                                       (3000, 313), (2000, 1001), (2000, 5001), (1100, 9001),
                                       (300000, 61), (17000, 1001), (3100, 7001)])
def test_gradients_of_many_odd_rows(rows, cols, dsum, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    h, dy = normal(g, rows, cols, dtype, 2.0, pad=2), normal(g, rows, cols, dtype, 0.5)
    ds = normal(g, rows, cols, dtype, 0.25, pad=0) if dsum else None
    w = weight(g, cols, dtype)
    inv = armx.rms_norm_rows(h, w, keep_inv_rms=True).inv_rms
    got = armx.rms_norm_rows_backward(dy, h, w, inv, dsum=ds)
    # each row's dx: as a row of a small batch, and by the formula
    at = spots(rows)
    lo = rows // 2
    for first, last in ((0, 300), (lo, lo + 300), (rows - 300, rows)):
        few = armx.rms_norm_rows_backward(dy[first:last], h[first:last], w, inv[first:last],
                                          dsum=None if ds is None else ds[first:last])
        assert np.array_equal(bits(got.dx[first:last]), bits(few.dx))
    dx, _, a, b, _ = layer.rms_norm_backward(f64(dy[at]), f64(h[at]), f64(w), f64(inv[at]),
                                             None if ds is None else f64(ds[at]))
    # roundings as for few rows: 4 on either term, the second's mean, squares and products
    # (6) and the row's sum, dsum's addition, then the type
    tol = (HALF[dtype] * np.abs(dx) + U * (4 * a + (10 + sum_depth(cols)) * b)
           + U * (np.abs(dx) if dsum else 0)) * 1.02 + FLOOR[dtype]
    assert np.all(np.abs(f64(got.dx[at]) - dx) <= tol)
    # dweight: two roundings a term, and the additions that it meets
    dw, size = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20000):
        n = dy[i:i + 20000].double() * h[i:i + 20000].double() * inv[i:i + 20000, None].double()
        dw += n.sum(0)
        size += n.abs().sum(0)
    tol = (dweight_depth(rows, cols) + 2) * U * 1.02 * size + 2.0 ** -149
    assert bool(((got.dweight.double() - dw).abs() <= tol).all())


# every form of dweight: columns apart (narrow, wide, past the registers, one round of rows
# and more), partial sums of 1 to 32 rows at a time, one block to all of them
@pytest.mark.parametrize("rows,cols", [(1, 1), (33, 5), (129, 300), (700, 2056), (1000, 4096),
                                       (300, 16384), (2600, 16390), (2100, 33000), (1500, 40001),
                                       (1025, 8), (1100, 61), (70000, 16), (600000, 16),
                                       (300000, 61), (40000, 101), (9000, 250), (20000, 313),
                                       (5000, 1000), (8192, 4096), (3000, 5001), (1025, 9000)])
def test_no_row_is_lost_from_dweight(rows, cols):
    # whole numbers and 1 / rms = 1: every sum stays below 2^24, so dweight is exact
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    dtype = torch.float16 if rows % 2 else torch.bfloat16
    h, dy = whole(g, rows, cols, dtype, 5), whole(g, rows, cols, dtype, 5, pad=0)
    one, w = torch.ones(rows, device="cuda"), torch.ones(cols, dtype=dtype, device="cuda")
    want = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20000):
        want += (dy[i:i + 20000].double() * h[i:i + 20000].double()).sum(0)
    for ds in (None, h):
        got = armx.rms_norm_rows_backward(dy, h, w, one, dsum=ds)
        assert torch.equal(got.dweight.double(), want)
    over = dy.clone() if dy.is_contiguous() else pitched(rows, cols, dtype).copy_(dy)
    got = armx.rms_norm_rows_backward(over, h, w, one, out=over)
    assert torch.equal(got.dweight.double(), want)


# rows * cols of 2^24 and more: results written past the caches
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(420000, 41), (170000, 101), (70000, 251), (40000, 509),
                                       (17000, 1001), (4200, 4099), (2100, 8195), (1050, 16390),
                                       (4096, 4096)])
def test_norms_and_codes_past_the_caches(rows, cols, dtype):
    assert rows * cols >= 1 << 24
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, r = normal(g, rows, cols, dtype, 2.0), normal(g, rows, cols, dtype, 1.0, pad=0)
    w = weight(g, cols, dtype)
    eps = 1e-5
    n = armx.rms_norm_rows(x, w, residual=r, eps=eps, keep_inv_rms=True)
    q = armx.rms_norm_rows_int8(x, w, residual=r, eps=eps)
    c = armx.quantize_rows_int8(x)
    plain = armx.rms_norm_rows(x, w, eps=eps)
    for first in (0, rows // 3, rows - 300):
        s = slice(first, first + 300)
        small = armx.rms_norm_rows(x[s], w, residual=r[s], eps=eps, keep_inv_rms=True)
        small8 = armx.rms_norm_rows_int8(x[s], w, residual=r[s], eps=eps)
        smallc = armx.quantize_rows_int8(x[s])
        for big, few in ((n.out, small.out), (n.sum, small.sum), (n.inv_rms, small.inv_rms),
                         (q.codes, small8.codes), (q.scales, small8.scales), (q.sum, small.sum),
                         (c.codes, smallc.codes), (c.scales, smallc.scales),
                         (plain.out, armx.rms_norm_rows(x[s], w, eps=eps).out)):
            assert np.array_equal(bits(big[s]), bits(few))
    at = spots(rows)
    h = n.sum[at]
    assert np.array_equal(bits(h), bits((x[at].float() + r[at].float()).to(dtype)))
    rel = check_norm(n.out[at], h, w, n.inv_rms[at], eps)
    _, inv = layer.rms_norm(f64(h), f64(w), eps)
    check_codes(q.codes[at], q.scales[at], f32(h) * f32(w), inv, rel)
    check_codes(c.codes[at], c.scales[at], f32(x[at]), 1.0, 0.0)
    # every value of what is exact: the sums, and the codes' largest
    for i in range(0, rows, 50000):
        s = slice(i, i + 50000)
        assert torch.equal(n.sum[s], (x[s].float() + r[s].float()).to(dtype))
        assert bool((c.codes[s].abs().amax(1) == 127).all())
        # (in 64 bits and rounded: the binary32 quotient; a binary32 division by a number
        # may be a product with its reciprocal)
        assert torch.equal(c.scales[s], (x[s].abs().amax(1).double() / 127).float())


# codes only: more rows than blocks, so that blocks walk on, on every layout of a row
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(300000, 61), (300000, 64), (140000, 128), (70001, 250),
                                       (35000, 500), (40000, 1000), (9000, 2041), (5000, 4096),
                                       (5003, 3999)])
def test_codes_of_more_rows_than_blocks(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = normal(g, rows, cols, dtype, 3.0)
    x[rows // 2] = 0.0
    x[rows - 2, cols - 1] = float("inf")
    q, s = armx.quantize_rows_int8(x)
    for first in range(0, rows, 1000):           # all of them, in small batches
        few = armx.quantize_rows_int8(x[first:first + 1000])
        assert torch.equal(q[first:first + 1000], few.codes)
        assert torch.equal(s[first:first + 1000].isnan(), few.scales.isnan())
        assert torch.equal(s[first:first + 1000].nan_to_num(-1), few.scales.nan_to_num(-1))
    at = spots(rows) + [rows // 2]
    check_codes(q[at], s[at], f32(x[at]), 1.0, 0.0)
    assert s[rows // 2] == 0 and s[rows - 2].isnan() and s.isnan().sum() == 1


def test_the_walk_of_the_codes():
    # the blocks that the longest of the walks above fills: what makes them walk on
    cu = torch.cuda.get_device_properties(0).multi_processor_count
    for rows, cols in ((300000, 61), (300000, 64), (140000, 128), (70001, 250), (35000, 500),
                       (40000, 1000), (9000, 2041), (5000, 4096), (5003, 3999)):
        chunks = -(-cols // 8)
        threads = 256 if chunks <= 64 else -(-chunks // 64) * 64
        assert -(-rows // rows_per_block(cols)) > cu * 32 * 256 // threads
