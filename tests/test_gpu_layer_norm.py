"""rms_norm_rows, rms_norm_rows_int8, quantize_rows_int8 and
rms_norm_rows_backward against the 64-bit oracle: every way a row can lie on
threads, odd widths, pitches, empty and single rows, zeros, infinities and NaN,
exact halves, in-place calls, batch invariance, graphs, streams and guards."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _layer import FLOOR, HALF, TYPES, U, f32, f64, ids, make, sum_depth
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def bits(t):
    return t.detach().cpu().contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[
        t.element_size()]).numpy()


def check_norm(y, h, w, inv, eps):
    """y and inv against the oracle on the sum h that was written."""
    want, want_inv = layer.rms_norm(f64(h), f64(w), eps)
    # inv: the sum's additions count half through the root; the quotient, eps,
    # the root and the division one rounding each (1.01: higher orders)
    rel_inv = (sum_depth(h.shape[1]) / 2 + 4) * U * 1.01
    if inv is not None:
        assert np.all(np.abs(f64(inv) - want_inv) <= rel_inv * want_inv)
    tol = np.abs(want) * (HALF[y.dtype] + rel_inv + 2 * U) * 1.01 + FLOOR[y.dtype]
    bad = np.abs(f64(y) - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], f64(y)[bad][:4], want[bad][:4])
    return rel_inv


def check_codes(q, s, p, inv, rel_inv):
    """Codes to the last one, scales within their few roundings; p the binary32
    products, inv the oracle's 1 / rms."""
    want, top = layer.codes(p)
    assert np.array_equal(q.cpu().numpy(), want)
    want_s = top * inv / 127
    got = f64(s)
    assert np.array_equal(np.isnan(got), np.isnan(want_s))
    # half the smallest binary32 step where a scale is subnormal
    assert np.all(np.abs(got - want_s)[~np.isnan(want_s)]
                  <= ((rel_inv + 2 * U) * 1.01 * want_s + 2.0 ** -149)[~np.isnan(want_s)])


# every row_shape (8 .. 64 lanes; whole wavefronts with 1, 2 or 4 chunks a lane; the
# loop) at its ends, odd widths among them
COLS = [1, 7, 8, 63, 64, 65, 128, 129, 250, 256, 257, 511, 512, 513, 1001, 1024, 1025, 2048,
        2049, 2056, 4096, 4097, 5001, 8192, 8193, 16384, 16391, 32768, 32769, 40000, 100003]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", COLS)
def test_norms_and_codes(cols, dtype):
    rng = np.random.default_rng(cols)
    rows = 37 if cols <= 4096 else 5
    eps = 1e-5
    for residual in (False, True):
        x = make(rng, rows, cols, dtype, 2.0, pad=1, device="cuda")
        r = make(rng, rows, cols, dtype, 1.0, pad=3, device="cuda") if residual else None
        w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).to(dtype).cuda()
        got = armx.rms_norm_rows(x, w, residual=r, eps=eps, keep_inv_rms=True)
        h = x
        if residual:
            h = got.sum
            assert np.array_equal(bits(h), bits((x.float() + r.float()).to(dtype)))
        else:
            assert got.sum is None
        rel = check_norm(got.out, h, w, got.inv_rms, eps)
        q = armx.rms_norm_rows_int8(x, w, residual=r, eps=eps)
        if residual:
            assert np.array_equal(bits(q.sum), bits(h))
        _, inv = layer.rms_norm(f64(h), f64(w), eps)
        check_codes(q.codes, q.scales, f32(h) * f32(w), inv, rel)
    c = armx.quantize_rows_int8(x)
    check_codes(c.codes, c.scales, f32(x), 1.0, 0.0)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (2, 64), (3, 8), (1000, 64), (4099, 136),
                                       (513, 2056), (300, 8192), (70000, 16), (33, 33000),
                                       (512, 1001), (513, 1024), (1024, 2049), (1025, 4100),
                                       (1200, 7000), (300, 16384), (520, 16390), (90, 32768)])
@pytest.mark.parametrize("dsum", [False, True])
def test_backward(rows, cols, dtype, dsum):
    rng = np.random.default_rng(rows + cols)
    h = make(rng, rows, cols, dtype, 2.0, pad=2, device="cuda")
    dy = make(rng, rows, cols, dtype, 0.5, pad=1, device="cuda")
    ds = make(rng, rows, cols, dtype, 0.25, device="cuda") if dsum else None
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).to(dtype).cuda()
    inv = armx.rms_norm_rows(h, w, keep_inv_rms=True).inv_rms
    got = armx.rms_norm_rows_backward(dy, h, w, inv, dsum=ds)
    check_backward(got, dy, h, w, inv, ds)


def check_backward(got, dy, h, w, inv, ds):
    rows, cols = h.shape
    dx, dw, a, b, c = layer.rms_norm_backward(f64(dy), f64(h), f64(w), f64(inv),
                                              None if ds is None else f64(ds))
    # dx: g, the difference and inv's product one rounding each on either term
    # (4); the second term also the sum's additions, its mean, inv^2 (2), the
    # product of the two and h's (6 more); dsum's addition; then the type
    dtype = h.dtype
    tol = (HALF[dtype] * np.abs(dx) + U * (4 * a + (10 + sum_depth(cols)) * b)
           + U * (0 if ds is None else np.abs(dx))) * 1.02 + FLOOR[dtype]
    bad = np.abs(f64(got.dx) - dx) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], f64(got.dx)[bad][:4], dx[bad][:4])
    # dweight: two roundings a term, and no term meets more than rows + 8 additions
    assert np.all(np.abs(f64(got.dweight) - dw) <= (rows + 10) * U * 1.02 * c + 2.0 ** -149)


def test_backward_against_differences_of_the_forward():
    # float16 in, float32 sums out through codes' scales would round; take the
    # forward's own result in 16 bits and a step that is exact in 16 bits
    rng = np.random.default_rng(5)
    h0 = torch.from_numpy(rng.integers(-64, 65, (6, 40)) / 16).half().cuda()
    w = torch.from_numpy(rng.integers(8, 25, 40) / 16).half().cuda()
    dy = torch.from_numpy(rng.integers(-16, 17, (6, 40)) / 16).half().cuda()
    inv = armx.rms_norm_rows(h0, w, keep_inv_rms=True).inv_rms
    got = f64(armx.rms_norm_rows_backward(dy, h0, w, inv).dx)
    d = 1 / 16
    for j in (0, 3, 17, 39):
        e = torch.zeros_like(h0)
        e[:, j] = d
        up, down = (f64(armx.rms_norm_rows(h0 + s * e, w).out) for s in (1, -1))
        diff = ((up - down) * f64(dy)).sum(1) / (2 * d)
        exact = (layer.rms_norm(f64(h0 + e), f64(w), 1e-6)[0]
                 - layer.rms_norm(f64(h0 - e), f64(w), 1e-6)[0])
        exact = (exact * f64(dy)).sum(1) / (2 * d)
        # the difference quotient's own curvature, taken from 64 bits, and the
        # 40 outputs' roundings (half a step each way) over the step
        slack = np.abs(exact - layer.rms_norm_backward(f64(dy), f64(h0), f64(w), f64(inv))[0][:, j])
        noise = (np.abs(f64(dy)) * np.maximum(np.abs(up), np.abs(down))).sum(1) * 2.0 ** -10 / (2 * d)
        assert np.all(np.abs(diff - got[:, j]) <= slack + noise + 2.0 ** -11 * np.abs(got[:, j]) + 1e-4)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_exact_halves_and_neighbours(dtype):
    # quotients that are halves exactly, and products next to them
    rng = np.random.default_rng(9)
    rows, cols = 64, 1000
    p = torch.from_numpy(rng.integers(-254, 255, (rows, cols)) * 0.5).to(dtype)
    p[:, 0] = 127
    p = (p.float() * 2.0 ** torch.from_numpy(rng.integers(-6, 7, (rows, 1)))).to(dtype)
    c = armx.quantize_rows_int8(p.cuda())
    check_codes(c.codes, c.scales, f32(p), 1.0, 0.0)
    # a weight makes products of 22 (16) bits: near halves of every kind
    x = torch.from_numpy(rng.integers(1, 2048 if dtype == torch.float16 else 256,
                                      (rows, cols)).astype(np.float32)).to(dtype).cuda()
    w = torch.from_numpy(rng.integers(1, 255, cols).astype(np.float32)).to(dtype).cuda()
    q = armx.rms_norm_rows_int8(x, w)
    _, inv = layer.rms_norm(f64(x), f64(w), 1e-6)
    check_codes(q.codes, q.scales, f32(x) * f32(w), inv, (sum_depth(cols) / 2 + 4) * U * 1.01)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [24, 600, 3000, 40000])
def test_rows_of_zeros_infinities_and_nan(cols, dtype):
    rng = np.random.default_rng(3)
    x = make(rng, 6, cols, dtype)
    x[0] = 0
    x[1, cols // 2] = float("inf")
    x[2, cols - 1] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = -0.0
    x = x.cuda()
    w = torch.ones(cols, dtype=dtype, device="cuda")
    got = armx.rms_norm_rows(x, w, eps=1e-6, keep_inv_rms=True)
    y = f64(got.out)
    assert np.all(y[[0, 4]] == 0) and np.all(np.abs(f64(got.inv_rms)[[0, 4]] - 1e3) < 1e-3)
    assert np.isnan(y[1, cols // 2]) and np.isnan(y[2]).all() and np.isnan(y[3, 0])
    assert np.all(y[1, :cols // 2] == 0) and np.isfinite(y[5]).all()
    check_norm(got.out[5:], x[5:], w, got.inv_rms[5:], 1e-6)
    for q, s in (armx.quantize_rows_int8(x), armx.rms_norm_rows_int8(x, w)[:2]):
        q, s = q.cpu().numpy(), f64(s)
        assert not q[:5].any() and np.isnan(s[1:4]).all() and np.all(s[[0, 4]] == 0)
        assert np.array_equal(q, layer.codes(f32(x))[0]) and s[5] > 0
    # eps = 0 on a row of zeros: 0 times an infinity, as the formula says
    assert np.isnan(f64(armx.rms_norm_rows(x[:1], w, eps=0.0).out)).all()


def test_extreme_magnitudes():
    # bfloat16 rows near both ends of binary32: codes keep their definition
    rng = np.random.default_rng(4)
    for scale in (2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 2.0 ** -70, 2.0 ** -63, 2.0 ** 100, 2.0 ** 125):
        x = (torch.from_numpy(rng.uniform(-1, 1, (8, 776)).astype(np.float32)) * scale).bfloat16()
        c = armx.quantize_rows_int8(x.cuda())
        check_codes(c.codes, c.scales, f32(x), 1.0, 0.0)
    # float16 subnormals
    x = torch.from_numpy(rng.integers(-5, 6, (8, 776)).astype(np.int16)).abs().view(torch.float16)
    c = armx.quantize_rows_int8(x.cuda())
    check_codes(c.codes, c.scales, f32(x), 1.0, 0.0)
    # the residual's addition overflows float16 into an infinity, and rounds
    # half to even once
    a = torch.full((2, 64), 65504.0, dtype=torch.float16, device="cuda")
    b = torch.full((2, 64), 2049.0, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    got = armx.rms_norm_rows(a, w, residual=b)
    assert torch.isinf(got.sum).all() and torch.isnan(got.out).all()
    q = armx.rms_norm_rows_int8(a, w, residual=b)
    assert torch.isnan(q.scales).all() and not q.codes.any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [40, 704, 4104, 40000])
def test_outputs_may_stand_where_inputs_did(cols, dtype):
    rng = np.random.default_rng(6)
    x, r = (make(rng, 9, cols, dtype, device="cuda") for _ in range(2))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).to(dtype).cuda()
    want = armx.rms_norm_rows(x, w, residual=r)
    want8 = armx.rms_norm_rows_int8(x, w, residual=r)
    alone = armx.rms_norm_rows(x, w)
    for swap in (False, True):
        x1, r1 = x.clone(), r.clone()
        o, s = (r1, x1) if swap else (x1, r1)
        got = armx.rms_norm_rows(x1, w, residual=r1, out=o, sum_out=s)
        assert got.out is o and got.sum is s
        assert np.array_equal(bits(o), bits(want.out)) and np.array_equal(bits(s), bits(want.sum))
        x1, r1 = x.clone(), r.clone()
        got = armx.rms_norm_rows_int8(x1, w, residual=r1, sum_out=x1 if swap else r1)
        assert np.array_equal(bits(got.sum), bits(want.sum))
        assert np.array_equal(bits(got.codes), bits(want8.codes))
    x1 = x.clone()
    assert np.array_equal(bits(armx.rms_norm_rows(x1, w, out=x1).out), bits(alone.out))
    inv = armx.rms_norm_rows(x, w, keep_inv_rms=True).inv_rms
    g = armx.rms_norm_rows_backward(r, x, w, inv, dsum=want.out)
    for k in range(2):
        dy, ds = r.clone(), want.out.clone()
        o = (dy, ds)[k]
        got = armx.rms_norm_rows_backward(dy, x, w, inv, dsum=ds, out=o)
        assert got.dx is o and np.array_equal(bits(o), bits(g.dx))
        assert np.array_equal(bits(got.dweight), bits(g.dweight))


@pytest.mark.parametrize("rows,cols", [(9, 40), (600, 2056), (3000, 1000), (70, 20000), (40, 40000)])
def test_gradients_where_everything_is_one_matrix(rows, cols):
    # dy, h and dsum the same matrix, or two of them, and dx written over it
    rng = np.random.default_rng(13)
    x, y = (make(rng, rows, cols, torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).bfloat16().cuda()
    inv = armx.rms_norm_rows(x, w, keep_inv_rms=True).inv_rms
    for dy, ds in ((x, x), (y, x), (x, y), (x, None)):
        want = armx.rms_norm_rows_backward(dy, x, w, inv, dsum=ds)
        one, other = x.clone(), y.clone()
        of = {id(x): one, id(y): other, id(None): None}
        got = armx.rms_norm_rows_backward(of[id(dy)], one, w, inv, dsum=of[id(ds)], out=one)
        assert got.dx is one
        assert np.array_equal(bits(got.dx), bits(want.dx))
        assert np.array_equal(bits(got.dweight), bits(want.dweight))


@pytest.mark.parametrize("cols", [8, 100, 1000, 2048, 5001, 33000])
def test_batch_invariance(cols):
    rng = np.random.default_rng(7)
    rows = 300 if cols <= 5001 else 40
    x, r, dy = (make(rng, rows, cols, torch.bfloat16, device="cuda") for _ in range(3))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).bfloat16().cuda()
    full = armx.rms_norm_rows(x, w, residual=r, keep_inv_rms=True)
    full8 = armx.rms_norm_rows_int8(x, w, residual=r)
    dx = armx.rms_norm_rows_backward(dy, full.sum, w, full.inv_rms).dx
    for lo, hi in ((0, 1), (rows - 1, rows), (3, 3 + 17), (5, rows)):
        part = armx.rms_norm_rows(x[lo:hi], w, residual=r[lo:hi], keep_inv_rms=True)
        part8 = armx.rms_norm_rows_int8(x[lo:hi], w, residual=r[lo:hi])
        pdx = armx.rms_norm_rows_backward(dy[lo:hi], part.sum, w, part.inv_rms).dx
        for a, b in ((part.out, full.out), (part.inv_rms, full.inv_rms), (part8.codes, full8.codes),
                     (part8.scales, full8.scales), (pdx, dx)):
            assert np.array_equal(bits(a), bits(b[lo:hi]))


def test_empty_sizes():
    for dtype in TYPES:
        e = torch.empty(0, 64, dtype=dtype, device="cuda")
        w = torch.ones(64, dtype=dtype, device="cuda")
        got = armx.rms_norm_rows(e, w, residual=e.clone(), keep_inv_rms=True)
        assert got.out.shape == (0, 64) and got.inv_rms.shape == (0,)
        assert armx.quantize_rows_int8(e).codes.shape == (0, 64)
        g = armx.rms_norm_rows_backward(e, e, w, got.inv_rms)
        assert g.dx.shape == (0, 64) and not g.dweight.any()
        z = torch.empty(5, 0, dtype=dtype, device="cuda")
        n = torch.empty(0, dtype=dtype, device="cuda")
        assert not armx.rms_norm_rows(z, n, keep_inv_rms=True).inv_rms.any()
        assert not armx.rms_norm_rows_int8(z, n).scales.any()
        q = armx.quantize_rows_int8(z)
        assert q.codes.shape == (5, 0) and not q.scales.any()
        g = armx.rms_norm_rows_backward(z, z, n, torch.ones(5, device="cuda"))
        assert g.dx.shape == (5, 0) and g.dweight.shape == (0,)


GUARD = 4096


def guarded(rows, cols, multiple, dtype):
    """A matrix between guard bands, padding and bands filled with 0x5A."""
    pitch = (-(-cols // multiple) + 1) * multiple
    size = torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((2 * GUARD + rows * pitch * size,), 0x5A, dtype=torch.uint8, device="cuda")
    m = buf[GUARD:GUARD + rows * pitch * size].view(dtype).view(rows, pitch)
    return buf, m[:, :cols]


def untouched(buf, m):
    """Whether all but the matrix's own values still holds the fill."""
    copy = buf.clone()
    size = m.element_size()
    rows, cols = m.shape
    body = copy[GUARD:copy.numel() - GUARD].view(rows, -1)
    body[:, :cols * size] = 0x5A
    return bool((copy == 0x5A).all().item())


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 61), (33, 1003), (7, 5001), (3, 33001), (900, 20)])
def test_nothing_but_the_rows_is_written(rows, cols):
    rng = np.random.default_rng(8)
    dtype = torch.float16
    x, r = (make(rng, rows, cols, dtype, pad=1, device="cuda") for _ in range(2))
    w = torch.ones(cols, dtype=dtype, device="cuda")
    (bo, o), (bs, s), (bd, d) = (guarded(rows, cols, 8, dtype) for _ in range(3))
    (bq, q), (bq2, q2) = (guarded(rows, cols, 16, torch.int8) for _ in range(2))
    (bc, c), (bc2, c2) = (guarded(1, rows, 1, torch.float32) for _ in range(2))
    got = armx.rms_norm_rows(x, w, residual=r, out=o, sum_out=s, keep_inv_rms=True)
    armx.rms_norm_rows_int8(x, w, residual=r, out=q, scales=c[0], sum_out=s)
    armx.quantize_rows_int8(x, out=q2, scales=c2[0])
    need = armx.workspace_bytes(armx.OP_RMS_BACKWARD, rows, cols)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    bw, dw = guarded(1, cols, 4, torch.float32)
    armx.rms_norm_rows_backward(r, s, w, got.inv_rms, dsum=x, out=d, dweight=dw[0],
                                workspace=ws[:need] if need else None)
    torch.cuda.synchronize()
    for b, m in ((bo, o), (bs, s), (bd, d), (bq, q), (bq2, q2), (bc, c), (bc2, c2), (bw, dw)):
        assert untouched(b, m)
    assert bool((ws[need:] == 0x5A).all().item())


def test_python_refusals_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    w = torch.zeros(64, dtype=torch.float16, device="cuda")
    s = torch.zeros(4, device="cuda")
    for bad in (w.bfloat16(), w[:32], w.cpu(), torch.zeros(64, 2, dtype=torch.float16, device="cuda")[:, 0], None):
        with pytest.raises(ValueError):
            armx.rms_norm_rows(x, bad)
    for bad in (x.bfloat16(), x[:2], x.cpu(), x[:, :32], x.t().contiguous().t()):
        with pytest.raises(ValueError):
            armx.rms_norm_rows(x, w, residual=bad)
        with pytest.raises(ValueError):
            armx.rms_norm_rows(x, w, out=bad)
        with pytest.raises(ValueError):
            armx.rms_norm_rows_backward(x, bad, w, s)
    with pytest.raises(ValueError):
        armx.rms_norm_rows(x.t(), torch.zeros(4, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        armx.rms_norm_rows(x, w, sum_out=x.clone())
    with pytest.raises(ValueError):
        armx.rms_norm_rows(x[0], w)
    with pytest.raises(ValueError):
        armx.rms_norm_rows_backward(x, x, w, s[:3])
    with pytest.raises(armx.ArmxError) as e:     # rows that start off 16 bytes
        armx.quantize_rows_int8(torch.zeros(4, 65, dtype=torch.float16, device="cuda"))
    assert e.value.name == "ARMX_ERR_ALIGN"
    with pytest.raises(armx.ArmxError) as e:     # one row for all: broadcast
        armx.quantize_rows_int8(x[:1].expand(4, 64))
    assert e.value.name == "ARMX_ERR_SHAPE"
    with pytest.raises(armx.ArmxError) as e:
        armx.rms_norm_rows(x, w, eps=-1.0)
    assert e.value.name == "ARMX_ERR_CONFIG"


def test_more_than_2_to_the_31_bytes_of_rows():
    # offsets past 32 bits: 600k rows of 4096 16-bit values are 4.9 GB
    rows, cols = 600_000, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    one = torch.randn(1000, cols, generator=g, device="cuda").half()
    x = one.repeat(600, 1)
    w = torch.ones(cols, dtype=torch.float16, device="cuda")
    small, big = armx.rms_norm_rows_int8(one, w), armx.rms_norm_rows_int8(x, w)
    for lo in (0, 262_000, 524_000, 599_000):
        assert torch.equal(big.codes[lo:lo + 1000], small.codes)
        assert torch.equal(big.scales[lo:lo + 1000], small.scales)
    del big
    y = armx.rms_norm_rows(x, w, keep_inv_rms=True)
    assert torch.equal(y.out[599_000:], armx.rms_norm_rows(one, w).out)
    d = armx.rms_norm_rows_backward(x, x, w, y.inv_rms)
    s = armx.rms_norm_rows_backward(one, one, w, y.inv_rms[:1000])
    assert torch.equal(d.dx[599_000:], s.dx)
    # 600 times the same rows; every partial sum is below the total, so
    # (rows + 10) U of it bounds any order
    assert float((d.dweight.double() / 600 / s.dweight.double() - 1).abs().max()) <= 2 * (rows + 10) * U


def test_narrow_rows_of_a_pitch_past_32_bit_offsets():
    # two rows 2^28 bytes apart and more: bits as with the rows side by side
    cols, pitch = 41, (1 << 27) + 8
    rng = np.random.default_rng(12)
    near = [make(rng, 3, cols, torch.bfloat16, device="cuda") for _ in range(3)]
    hold = torch.zeros(2 * pitch + 192, dtype=torch.bfloat16, device="cuda")
    x, r, dy = (torch.as_strided(hold, (3, cols), (pitch, 1), 64 * i) for i in range(3))
    for a, b in zip((x, r, dy), near):
        a.copy_(b)
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).bfloat16().cuda()
    far = armx.rms_norm_rows(x, w, residual=r, keep_inv_rms=True)
    want = armx.rms_norm_rows(near[0], w, residual=near[1], keep_inv_rms=True)
    for a, b in zip(far, want):
        assert np.array_equal(bits(a), bits(b))
    for a, b in zip(armx.rms_norm_rows_int8(x, w, residual=r),
                    armx.rms_norm_rows_int8(near[0], w, residual=near[1])):
        assert np.array_equal(bits(a), bits(b))
    for a, b in zip(armx.rms_norm_rows_backward(dy, x, w, far.inv_rms, dsum=r),
                    armx.rms_norm_rows_backward(near[2], near[0], w, want.inv_rms, dsum=near[1])):
        assert np.array_equal(bits(a), bits(b))
