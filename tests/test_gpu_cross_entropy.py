"""cross_entropy_rows and cross_entropy_rows_backward against the 64-bit oracle: every
tile, odd sizes, pitches with NaN behind the rows, one row, one word, one value, ignored
and foreign targets, sums that are exact, several pieces, both results apart, batch
invariance, 64-bit places and guards."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import training

from _layer import FLOOR, HALF, TYPES, U, f64, ids, make
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def inputs(rng, rows, vocab, cols, dtype, ignored=0.2):
    x = make(rng, rows, cols, dtype, 1.0, pad=1, device="cuda")
    w = make(rng, vocab, cols, dtype, cols ** -0.5, pad=2, device="cuda")
    t = rng.integers(0, vocab, rows)
    t[rng.random(rows) < ignored] = -100
    return x, w, torch.from_numpy(t).cuda()


def e_logits(x, w):
    """How far a logit may be off: its products are exact in binary32, and each of its
    cols additions cuts off less than a unit, 2 U, of the sum of magnitudes."""
    return 2 * U * 1.02 * (x.shape[1] + 8) * (np.abs(f64(x)) @ np.abs(f64(w)).T)


def check_loss(got, x, w, t, exact_logits=False, ignore=-100):
    loss, lse, z = training.cross_entropy(f64(x), f64(w), t.cpu().numpy(), ignore)
    e_z = 0.0 * z if exact_logits else e_logits(x, w)
    # An exponential: the difference and its product with log2 e one rounding each, both
    # on an exponent of at most the row's range, the constant's own, and the instruction's
    # unit; then the joined sums' factors alike.  A sum of 64 has 6 additions, 8 + 16 and
    # one per 128 pieces follow; the logarithm is good to 2 units.  exp(z - lse) weighs
    # logits' errors, so no sum is off by more than the largest.
    span = z.max(1) - z.min(1)
    rel = U * (2 * (3 * span + 4) + 30 + w.shape[0] / 64 / 128)
    e_lse = (rel + e_z.max(1) + U * (4 * np.abs(np.log(w.shape[0])) + 4 + 2 * np.abs(lse))) * 1.02
    assert np.all(np.abs(f64(got.lse) - lse) <= e_lse), np.abs(f64(got.lse) - lse).max()
    assert np.array_equal(np.isnan(f64(got.loss)), np.isnan(loss))
    fine = ~np.isnan(loss)
    tn = t.cpu().numpy()
    hit = np.where((tn >= 0) & (tn < w.shape[0]), tn, 0)
    e_hit = e_z[np.arange(len(tn)), hit]
    bad = np.abs(f64(got.loss) - loss) > (e_lse + e_hit + U * np.abs(loss)) * 1.02
    assert not bad[fine].any(), np.abs(f64(got.loss) - loss)[fine].max()
    assert not f64(got.loss)[tn == ignore].any()


def check_grads(got, dloss, x, w, t, lse, exact_logits=False, ignore=-100):
    rows, cols = x.shape
    tn, g = t.cpu().numpy(), f64(dloss)
    live = tn != ignore
    xs = np.where(live[:, None], f64(x), 0.0)
    dx, dw, dz = training.cross_entropy_backward(g, f64(x), f64(w), tn, f64(lse), ignore)
    g = np.where(live, g, 0.0)
    ag = np.abs(g)[:, None]
    z = xs @ f64(w).T
    p = np.exp(z - f64(lse)[:, None]) * live[:, None]
    # exp(z - lse): the logit, lse times log2 e and the product's roundings on the
    # exponent, and the instruction's unit; the target's 1 one more on what is left
    e_z = 0.0 * z if exact_logits else 2 * U * 1.02 * (cols + 8) * (np.abs(xs) @ np.abs(f64(w)).T)
    e_p = p * (e_z + U * (3 * np.abs(z) + 3 * np.abs(f64(lse))[:, None] + 4)) + U * np.abs(p)
    half, floor = HALF[x.dtype], FLOOR[x.dtype]
    # A value of dz is rounded to 16 bits behind two products with scales (3 U).  Where
    # binary16's are small they are cut at its smallest step: dx's are scaled to 2^14 over
    # the row's 1 - p of its target (at least 2^-14), dweight's to 2^15 over the largest |g|.
    aw, ax, adz = np.abs(f64(w)), np.abs(xs), np.abs(dz)
    if got.dx is not None:
        rest = np.maximum(np.abs(dz).max(1) / np.where(g == 0, 1, np.abs(g)), 2.0 ** -14)[:, None]
        e_dz = adz * (half + 3 * U) + ag * e_p + floor * ag * rest * 2.0 ** -13
        tol = e_dz @ aw + 2 * U * (w.shape[0] + 40) * (adz @ aw)
        bad = ~(np.abs(f64(got.dx) - dx) <= (tol + half * (np.abs(dx) + tol)) * 1.02 + floor)
        assert not bad.any(), (np.argwhere(bad)[:4], f64(got.dx)[bad][:4], dx[bad][:4])
        assert not f64(got.dx)[~live].any()
    if got.dweight is not None:
        # up to 128 rows a second term holds what the first one's rounding leaves
        once = half if rows > 128 else half ** 2
        e_dz = adz * (once + 4 * U) + ag * e_p + floor * np.abs(g).max() * 2.0 ** -15
        tol = e_dz.T @ ax + 2 * U * (2 * rows + 40) * (adz.T @ ax)
        last, least = (half, floor) if got.dweight.dtype == x.dtype else (U, 2.0 ** -149)
        bad = ~(np.abs(f64(got.dweight) - dw) <= (tol + last * (np.abs(dw) + tol)) * 1.02 + least)
        assert not bad.any(), (np.argwhere(bad)[:4], f64(got.dweight)[bad][:4], dw[bad][:4])


def run_both(rng, x, w, t, exact_logits=False, **kw):
    got = armx.cross_entropy_rows(x, w, t, **kw)
    check_loss(got, x, w, t, exact_logits, **({} if "ignore_index" not in kw else
                                              {"ignore": kw["ignore_index"]}))
    dloss = torch.from_numpy(rng.uniform(0.5, 1.5, x.shape[0]).astype(np.float32)).cuda()
    if t.numel():
        dloss[0] = -2.0   # any sign and size
    grads = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse, **kw)
    check_grads(grads, dloss, x, w, t, got.lse, exact_logits,
                **({} if "ignore_index" not in kw else {"ignore": kw["ignore_index"]}))
    return got, grads, dloss


SHAPES = [(1, 1, 1), (1, 2, 8), (1, 1000, 64), (3, 65, 7), (16, 128, 64), (17, 129, 65), (31, 1001, 100),
          (33, 300, 1000), (64, 64, 128), (65, 1025, 129), (127, 500, 33), (128, 700, 200),
          (129, 700, 201), (130, 2001, 72), (200, 3000, 130), (257, 257, 257), (300, 5000, 64),
          (513, 700, 513), (700, 2500, 320), (1030, 1100, 136), (2, 40000, 24), (70, 33, 2056)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,vocab,cols", SHAPES)
def test_against_64_bits(rows, vocab, cols, dtype):
    rng = np.random.default_rng(rows + vocab + cols)
    run_both(rng, *inputs(rng, rows, vocab, cols, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,vocab,cols", [(5, 300, 512), (40, 1000, 1000), (150, 500, 64),
                                             (600, 1200, 96), (300, 300, 2000)])
def test_logits_that_are_exact(rows, vocab, cols, dtype):
    # quarters: every sum of their products is exact in binary32, so that only the
    # exponentials and their sums are rounded
    rng = np.random.default_rng(cols)
    x = make(rng, rows, cols, dtype, device="cuda")
    w = make(rng, vocab, cols, dtype, device="cuda")
    x.copy_(torch.from_numpy(rng.integers(-3, 4, (rows, cols)) / 4))
    w.copy_(torch.from_numpy(rng.integers(-1, 2, (vocab, cols)) / 4))
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    run_both(rng, x, w, t, exact_logits=True)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_rows_that_are_sure_of_their_target(dtype):
    # 1 - p from near 1 down to nothing at all
    rng = np.random.default_rng(8)
    x, w, t = inputs(rng, 200, 400, 256, dtype, 0.0)
    sure = torch.linspace(0, 40, 200, device="cuda")[:, None]
    x.copy_(x.float() + sure * w[t].float())
    run_both(rng, x, w, t)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows", [9, 140])
def test_ignored_and_foreign_targets(rows, dtype):
    rng = np.random.default_rng(rows)
    vocab, cols = 700, 136
    x, w, t = inputs(rng, rows, vocab, cols, dtype)
    t[1], t[rows // 2] = 0, vocab - 1
    # whatever stands in ignored rows, and in their gradient, reaches nothing
    t[2] = t[5] = -100
    dirty = x.clone()
    wide = torch.empty(rows, 160, dtype=dtype, device="cuda")[:, :cols]
    wide.copy_(dirty)
    wide[2], wide[5] = float("nan"), float("inf")
    got = armx.cross_entropy_rows(wide, w, t)
    want = armx.cross_entropy_rows(x, w, t)
    rest = [i for i in range(rows) if i not in (2, 5)]
    assert torch.equal(got.loss, want.loss) and torch.equal(got.lse[rest], want.lse[rest])
    dloss = torch.ones(rows, device="cuda")
    clean = armx.cross_entropy_rows_backward(dloss, x, w, t, want.lse)
    dloss[2], dloss[5] = float("nan"), float("inf")
    grads = armx.cross_entropy_rows_backward(dloss, wide, w, t, got.lse)
    assert torch.equal(grads.dx, clean.dx) and torch.equal(grads.dweight, clean.dweight)
    assert not grads.dx[[2, 5]].any()
    # another index to ignore, which is a word of the vocabulary
    run_both(rng, x, w, torch.where(t == -100, 3, t), ignore_index=3)
    # a target outside the vocabulary
    for foreign in (vocab, -1, 1 << 40, -(1 << 40)):
        t2 = t.clone()
        t2[4] = foreign
        got = armx.cross_entropy_rows(x, w, t2)
        assert torch.isnan(got.loss[4]) and not torch.isnan(got.loss[5:]).any()
        assert torch.equal(got.lse, want.lse)
        grads = armx.cross_entropy_rows_backward(torch.ones(rows, device="cuda"), x, w, t2, got.lse)
        others = [i for i in range(rows) if i != 4]
        assert torch.isnan(grads.dx[4]).all() and torch.isnan(grads.dweight).all()
        assert torch.equal(grads.dx[others], clean.dx[others])
    all_ignored = torch.full_like(t, -100)
    got = armx.cross_entropy_rows(x, w, all_ignored)
    assert not got.loss.any() and torch.equal(got.lse, want.lse)
    grads = armx.cross_entropy_rows_backward(dloss, x, w, all_ignored, got.lse)
    assert not grads.dx.any() and not grads.dweight.any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_what_is_not_finite(dtype):
    rng = np.random.default_rng(4)
    x, w, t = inputs(rng, 50, 300, 64, dtype, 0.0)
    x[7, 3], x[9, 60] = float("nan"), float("inf")
    got = armx.cross_entropy_rows(x, w, t)
    fine = [i for i in range(50) if i not in (7, 9)]
    assert torch.isnan(got.loss[[7, 9]]).all() and torch.isfinite(got.loss[fine]).all()
    # words that cannot be: their logits are minus infinity
    x, w, t = inputs(rng, 50, 300, 64, dtype, 0.0)
    x[:, 0] = 1.0
    t.clamp_(max=99)
    open_ = armx.cross_entropy_rows(x, w[:100], t)
    w[100:] = 0.0
    w[100:, 0] = -float("inf")
    got = armx.cross_entropy_rows(x, w, t)
    # the same sums, in pieces that are cut off elsewhere
    assert np.all(np.abs(f64(got.loss) - f64(open_.loss)) <= 1e-5)
    # a loss gradient of infinity or NaN
    for bad in (float("inf"), float("nan")):
        dloss = torch.ones(50, device="cuda")
        dloss[3] = bad
        g = armx.cross_entropy_rows_backward(dloss, x, w[:100], t, open_.lse)
        others = [i for i in range(50) if i != 3]
        assert torch.isfinite(g.dx[others]).all() and torch.isnan(g.dx[3]).all()
        assert torch.isnan(g.dweight).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_gradients_of_any_size(dtype):
    rng = np.random.default_rng(6)
    for rows in (20, 200):
        x, w, t = inputs(rng, rows, 500, 64, dtype, 0.1)
        lse = armx.cross_entropy_rows(x, w, t).lse
        for size in (2.0 ** -20, 2.0 ** 12):
            dloss = torch.from_numpy(rng.uniform(0.5, 1.5, rows) * size).float().cuda()
            got = armx.cross_entropy_rows_backward(dloss, x, w, t, lse, dweight_dtype=torch.float32)
            check_grads(got, dloss, x, w, t, lse)
        zero = torch.zeros(rows, device="cuda")
        got = armx.cross_entropy_rows_backward(zero, x, w, t, lse)
        assert not got.dx.any() and not got.dweight.any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,vocab,cols", [(70, 900, 100), (300, 1000, 333)])
def test_results_apart_and_in_32_bits(rows, vocab, cols, dtype):
    rng = np.random.default_rng(cols)
    x, w, t = inputs(rng, rows, vocab, cols, dtype)
    lse = armx.cross_entropy_rows(x, w, t).lse
    dloss = torch.rand(rows, device="cuda")
    both = armx.cross_entropy_rows_backward(dloss, x, w, t, lse)
    a = armx.cross_entropy_rows_backward(dloss, x, w, t, lse, need_dweight=False)
    b = armx.cross_entropy_rows_backward(dloss, x, w, t, lse, need_dx=False,
                                         dweight_dtype=torch.float32)
    assert a.dweight is None and torch.equal(a.dx, both.dx)
    assert b.dx is None and b.dweight.dtype == torch.float32
    check_grads(b, dloss, x, w, t, lse)
    # the same sums times the same factor: in 16 bits the product is rounded to half a
    # step, once (the multiplication's result need not pass through 32 bits), in 32 by U
    off = (both.dweight.double() - b.dweight.double()).abs()
    assert torch.all(off <= (HALF[dtype] + 2 * U) * b.dweight.double().abs() + FLOOR[dtype])


def test_a_row_does_not_depend_on_the_others():
    # its loss has the same bits in every batch, that is in every tile
    rng = np.random.default_rng(2)
    for cols, vocab in ((100, 1000), (1024, 3001)):
        x, w, t = inputs(rng, 1500, vocab, cols, torch.bfloat16, 0.0)
        want = armx.cross_entropy_rows(x, w, t)
        for n in (1, 2, 16, 17, 33, 65, 130, 300, 700):
            got = armx.cross_entropy_rows(x[100:100 + n], w, t[100:100 + n])
            assert torch.equal(got.loss, want.loss[100:100 + n]), n
            assert torch.equal(got.lse, want.lse[100:100 + n]), n


def test_several_pieces():
    # 2^27 values of dz at a time: 65536 rows of a vocabulary past one piece's 2048
    rng = np.random.default_rng(9)
    rows, vocab, cols = 65536 + 8, 4500, 16
    x, w, t = inputs(rng, rows, vocab, cols, torch.float16)
    got = armx.cross_entropy_rows(x, w, t)
    dloss = torch.rand(rows, device="cuda")
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse, dweight_dtype=torch.float32)
    some = torch.from_numpy(np.r_[0:300, rows - 300:rows]).cuda()
    part = armx.CrossEntropyGrads(g.dx[some], None)
    check_loss(armx.CrossEntropy(got.loss[some], got.lse[some]), x[some], w, t[some])
    check_grads(part, dloss[some], x[some], w, t[some], got.lse[some])
    # dweight of all rows: batches of rows, added up in 64 bits
    dw, tol = 0.0, 0.0
    for at in range(0, rows, 8192):
        s = slice(at, at + 8192)
        _, d, dz = training.cross_entropy_backward(f64(dloss[s]), f64(x[s]), f64(w),
                                                   t[s].cpu().numpy(), f64(got.lse[s]))
        dw = dw + d
        live = (t[s] != -100).cpu().numpy()[:, None]
        tol = tol + np.abs(dz).T @ (np.abs(f64(x[s])) * live)
    # a rounding of dz, its logit's and exponential's (below 2^-13 together here), and
    # the additions
    assert np.all(np.abs(f64(g.dweight) - dw) <= tol * (2.0 ** -11 + 2.0 ** -13 + 2 * U * rows))


def test_pieces_in_parts():
    # two pieces of 2^27 values of dz and a little more, each with its product for dx in
    # parts, the last of them shorter or empty in the second piece
    rng = np.random.default_rng(10)
    rows, vocab, cols = 3000, 50001, 72
    x, w, t = inputs(rng, rows, vocab, cols, torch.bfloat16)
    got = armx.cross_entropy_rows(x, w, t)
    dloss = torch.from_numpy(rng.uniform(0.5, 1.5, rows).astype(np.float32)).cuda()
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse, dweight_dtype=torch.float32)
    some = torch.from_numpy(np.r_[0:60, rows - 60:rows]).cuda()
    check_grads(armx.CrossEntropyGrads(g.dx[some], None), dloss[some], x[some], w, t[some],
                got.lse[some])
    # dweight's rows at the pieces' ends and those of some targets, with check_grads' bound
    tn, lse, xs = t.cpu().numpy(), f64(got.lse), f64(x)
    live = tn != -100
    words = np.unique(np.r_[0:40, 25000:25200, vocab - 40:vocab, tn[live][:40]])
    ws = f64(w)[words]
    z, ag = xs @ ws.T, (f64(dloss) * live)[:, None]
    p = np.exp(z - lse[:, None])
    dz = (p - (tn[:, None] == words)) * ag
    e_z = 2 * U * 1.02 * (cols + 8) * (np.abs(xs) @ np.abs(ws).T)
    e_p = p * (e_z + U * (3 * np.abs(z) + 3 * np.abs(lse)[:, None] + 5))
    e_dz = np.abs(dz) * (HALF[x.dtype] + 4 * U) + ag * e_p + FLOOR[x.dtype] * ag.max() * 2.0 ** -15
    tol = e_dz.T @ np.abs(xs) + 2 * U * (2 * rows + 40) * (np.abs(dz).T @ np.abs(xs))
    want = dz.T @ xs
    assert np.all(np.abs(f64(g.dweight)[words] - want) <= (tol + U * np.abs(want)) * 1.02)


def test_places_past_32_bits():
    vocab, cols = (1 << 19) + 13, 4096 + 8   # 2^31 values and more
    w = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda")
    w.normal_(std=cols ** -0.5)
    x = torch.randn(3, cols, device="cuda").bfloat16()
    t = torch.tensor([vocab - 1, 5, vocab - 300], device="cuda")
    z = torch.cat([x.double() @ w[v:v + 65536].double().t().contiguous()
                   for v in range(0, vocab, 65536)], 1)
    lse = torch.logsumexp(z, 1)
    got = armx.cross_entropy_rows(x, w, t)
    # as above: the logits' bound, at the sum of magnitudes that such rows have
    bound = 2 * U * (cols + 8) * float((x.double().abs() @ w[:4096].double().abs().t().contiguous()).max()) * 1.5
    assert torch.all((got.lse.double() - lse).abs() <= bound + 1e-5)
    assert torch.all((got.loss.double() - (lse - z.gather(1, t[:, None])[:, 0])).abs() <= 2 * bound + 1e-5)
    dloss = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    g = armx.cross_entropy_rows_backward(dloss, x, w, t, got.lse)
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(3), t] -= 1
    dz *= dloss[:, None]
    for rows in (slice(0, 64), slice(vocab - 320, vocab)):
        want = dz[:, rows].t().contiguous() @ x.double()
        assert torch.all((g.dweight[rows].double() - want).abs() <=
                         (HALF[torch.bfloat16] * 1.1 + 4 * bound) * (dz[:, rows].abs().t().contiguous()
                                                                    @ x.double().abs()))
    want = sum(dz[:, v:v + 65536] @ w[v:v + 65536].double() for v in range(0, vocab, 65536))
    top = sum(dz[:, v:v + 65536].abs() @ w[v:v + 65536].double().abs() for v in range(0, vocab, 65536))
    assert torch.all((g.dx.double() - want).abs() <= (2 * HALF[torch.bfloat16] * 1.1 + 4 * bound) * top)


def test_results_stay_inside():
    rng = np.random.default_rng(3)
    for rows, vocab, cols in ((5, 13, 9), (150, 300, 100), (300, 700, 129)):
        mark = 55.0
        x, w, t = inputs(rng, rows, vocab, cols, torch.float16)
        pitch = -(-cols // 8) * 8 + 8
        dx, dw = (torch.full((n + 2, pitch), mark, dtype=torch.float16, device="cuda")
                  for n in (rows, vocab))
        dw32 = torch.full((vocab + 2, pitch), mark, device="cuda")
        side = torch.full((2, rows + 8), mark, device="cuda")
        got = armx.cross_entropy_rows(x, w, t, loss=side[0, 4:4 + rows], lse=side[1, 4:4 + rows])
        assert (side[:, :4] == mark).all() and (side[:, 4 + rows:] == mark).all()
        check_loss(got, x, w, t)
        dloss = torch.rand(rows, device="cuda")
        lse = got.lse.clone()
        for d in (dw, dw32):
            g = armx.cross_entropy_rows_backward(dloss, x, w, t, lse, out=dx[1:-1, :cols],
                                                 dweight=d[1:-1, :cols])
            check_grads(g, dloss, x, w, t, lse)
            for m in (dx, d):
                m[1:-1, :cols].fill_(mark)
                assert (m == mark).all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(100, 64, dtype=torch.bfloat16, device="cuda")
    t, none = torch.empty(0, dtype=torch.long, device="cuda"), torch.empty(0, device="cuda")
    got = armx.cross_entropy_rows(x, w, t)
    assert got.loss.shape == got.lse.shape == (0,)
    for dtype in (torch.bfloat16, torch.float32):
        dw = torch.ones(100, 72, dtype=dtype, device="cuda")
        g = armx.cross_entropy_rows_backward(none, x, w, t, none, dweight=dw[:, :64])
        assert g.dx.shape == (0, 64) and not dw[:, :64].any() and (dw[:, 64:] == 1).all()


def test_refused_on_the_gpu():
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    w = torch.zeros(100, 64, dtype=torch.float16, device="cuda")
    t, f = torch.zeros(4, dtype=torch.long, device="cuda"), torch.zeros(4, device="cuda")
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    back = armx.cross_entropy_rows_backward
    for call, error, match in [
            (lambda: armx.cross_entropy_rows(x, w.bfloat16(), t), ValueError, "weight"),
            (lambda: armx.cross_entropy_rows(x, w[:, :63], t), ValueError, "weight"),
            (lambda: armx.cross_entropy_rows(x, w, t.int()), ValueError, "targets"),
            (lambda: armx.cross_entropy_rows(x, w, t[:3]), ValueError, "targets"),
            (lambda: armx.cross_entropy_rows(x, w, t.cpu()), ValueError, "targets"),
            (lambda: armx.cross_entropy_rows(x, w, t, ignore_index=1.5), TypeError, "ignore_index"),
            (lambda: armx.cross_entropy_rows(x, w, t, ignore_index=1 << 63), TypeError, "ignore_index"),
            (lambda: armx.cross_entropy_rows(x, w[:0], t), armx.ArmxError, "SHAPE"),
            (lambda: armx.cross_entropy_rows(x, w, t, workspace=small[:16]), armx.ArmxError,
             "WORKSPACE"),
            (lambda: armx.cross_entropy_rows(x, w, t, workspace=small.cpu()), ValueError, "workspace"),
            (lambda: back(f.half(), x, w, t, f), ValueError, "dloss"),
            (lambda: back(f, x, w, t, f[:2]), ValueError, "lse"),
            (lambda: back(f, x, w, t, f, need_dx=False, need_dweight=False), ValueError, "wanted"),
            (lambda: back(f, x, w, t, f, need_dx=False, out=x), ValueError, "wanted"),
            (lambda: back(f, x, w, t, f, dweight_dtype=torch.bfloat16), TypeError, "dweight is"),
            (lambda: back(f, x, w, t, f, dweight_dtype=torch.float64), TypeError, "dweight is"),
            (lambda: back(f, x, w, t, f, dweight=w.bfloat16()), TypeError, "dweight is"),
            (lambda: back(f, x, w, t, f, workspace=small), armx.ArmxError, "WORKSPACE")]:
        with pytest.raises(error, match=match):
            call()
