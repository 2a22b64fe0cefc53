"""matmul_int8 bit for bit: the integer sums are exact and each later step is one
binary32 rounding, so numpy gives the same bits.  Sizes around every tile, odd
lengths, pitches whose padding holds codes, single tokens, empty sizes, the
extreme codes and lengths, graphs and guards."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _layer import ids, make_codes
from _parity import require_gpu

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def scales(rng, n):
    return torch.from_numpy(np.exp2(rng.uniform(-12, -4, n)).astype(np.float32)).cuda()


def expected(a, sa, b, sb, bias, dtype):
    """The documented roundings, on the CPU."""
    acc = torch.from_numpy(layer.product(a.cpu().numpy(), b.cpu().numpy())).float()
    y = acc * (sa.cpu()[:, None] * sb.cpu()[None, :])
    if bias is not None:
        y = y + bias.cpu().float()
    return y.to(dtype)


def same(got, want):
    view = torch.int32 if got.dtype == torch.float32 else torch.int16
    return torch.equal(got.cpu().contiguous().view(view), want.contiguous().view(view))


def run_case(m, n, k, dtype, bias, seed=0, pad=1):
    rng = np.random.default_rng([m, n, k, seed])
    a, b = make_codes(rng, m, k, pad, "cuda"), make_codes(rng, n, k, pad, "cuda")
    sa, sb = scales(rng, m), scales(rng, n)
    bi = torch.from_numpy(rng.standard_normal(n)).to(dtype).cuda() if bias else None
    got = armx.matmul_int8(a, sa, b, sb, bias=bi, dtype=dtype)
    assert got.shape == (m, n) and got.dtype == dtype
    assert same(got, expected(a, sa, b, sb, bi, dtype)), (m, n, k, dtype, bias)


@pytest.mark.parametrize("m", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128,
                               129, 192, 255, 256, 257, 300])
def test_row_counts(m):
    run_case(m, 272, 320, torch.bfloat16, m % 2 == 0)


@pytest.mark.parametrize("n", [1, 3, 4, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255,
                               256, 257, 1000])
def test_column_counts(n):
    for m in (1, 7, 40, 150):
        run_case(m, n, 256, torch.float16, n % 2 == 0)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257,
                               500, 512, 513, 1000, 1023, 1024, 1025, 4099])
def test_lengths(k):
    for m, n in ((1, 40), (20, 70), (130, 131), (260, 257)):
        run_case(m, n, k, torch.float32, k % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 4096, 4096), (5, 1003, 2049), (33, 1024, 4096),
                                   (64, 200, 8192), (129, 513, 1030), (513, 770, 640),
                                   (1030, 1028, 300), (2048, 1500, 128)])
def test_types_and_shapes(m, n, k, dtype):
    for bias in (False, True):
        run_case(m, n, k, dtype, bias, pad=0)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    m, n, k = (int(np.exp(rng.uniform(0, np.log(top)))) for top in (1500, 1500, 6000))
    run_case(m, n, k, DTYPES[seed % 3], seed % 2 == 0, seed, pad=int(rng.integers(0, 3)))


@pytest.mark.parametrize("m,n", [(1, 64), (17, 100), (130, 300)])
def test_the_largest_sums(m, n):
    # 131071 products of (-128)^2 stay below 2^31; opposite signs reach its other end
    k = 131071
    for va, vb in ((-128, -128), (-128, 127), (127, 127)):
        a = torch.full((m, k + 1), va, dtype=torch.int8, device="cuda")[:, :k]
        b = torch.full((n, k + 1), vb, dtype=torch.int8, device="cuda")[:, :k]
        one = torch.ones(max(m, n), device="cuda")
        got = armx.matmul_int8(a, one[:m], b, one[:n], dtype=torch.float32)
        assert torch.all(got == float(np.float32(k * va * vb)))


def test_batch_invariance():
    rng = np.random.default_rng(1)
    a, b = make_codes(rng, 600, 1111, 0, "cuda"), make_codes(rng, 700, 1111, 0, "cuda")
    sa, sb = scales(rng, 600), scales(rng, 700)
    full = armx.matmul_int8(a, sa, b, sb)
    for lo, hi in ((0, 1), (5, 9), (100, 117), (3, 70), (10, 140), (0, 400)):
        assert torch.equal(armx.matmul_int8(a[lo:hi], sa[lo:hi], b, sb), full[lo:hi])
        assert torch.equal(armx.matmul_int8(a, sa, b[lo:hi], sb[lo:hi]), full[:, lo:hi])


def test_special_scales():
    rng = np.random.default_rng(2)
    a, b = make_codes(rng, 6, 100, 0, "cuda"), make_codes(rng, 40, 100, 0, "cuda")
    sa, sb = scales(rng, 6), scales(rng, 40)
    sa[1], sa[2], sa[3] = 0.0, float("nan"), float("inf")
    a[0] = 0
    a[3] = 0
    got = armx.matmul_int8(a, sa, b, sb, dtype=torch.float32)
    assert not got[0].any() and not got[1].any()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()   # 0 times an infinity
    assert torch.isfinite(got[4:]).all()


def test_empty_sizes():
    one = torch.ones(64, device="cuda")
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    assert armx.matmul_int8(q[:0], one[:0], q, one[:4]).shape == (0, 4)
    assert armx.matmul_int8(q, one[:4], q[:0], one[:0]).shape == (4, 0)
    e = torch.empty(4, 0, dtype=torch.int8, device="cuda")
    bias = torch.arange(4, dtype=torch.float16, device="cuda")
    assert torch.equal(armx.matmul_int8(e, one[:4], e, one[:4], bias=bias), bias.expand(4, 4))
    assert not armx.matmul_int8(e, one[:4], e, one[:4]).any()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("m,n", [(1, 5), (3, 33), (40, 130), (200, 259)])
def test_pitched_output_between_guards(m, n, dtype):
    rng = np.random.default_rng(3)
    k = 333
    a, b = make_codes(rng, m, k, 2, "cuda"), make_codes(rng, n, k, 1, "cuda")
    sa, sb = scales(rng, m), scales(rng, n)
    want = expected(a, sa, b, sb, None, dtype)
    for pitch in (n, n + 1, (n + 3) // 4 * 4 + 4):
        for skew in (0, 1):      # an out that starts at any whole value
            buf = torch.full((64 + m * pitch + 64,), 77.0, dtype=dtype, device="cuda")
            out = torch.as_strided(buf, (m, n), (pitch, 1), 64 + skew)
            armx.matmul_int8(a, sa, b, sb, out=out)
            assert same(out, want), (pitch, skew)
            rest = buf.clone()
            torch.as_strided(rest, (m, n), (pitch, 1), 64 + skew).fill_(77.0)
            assert bool((rest == 77.0).all().item()), (pitch, skew)


def test_python_refusals_on_the_gpu():
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    for bad in (dict(a=q.t()), dict(b=q[:, :16]), dict(b=q.cpu()), dict(a_scales=s[:3]),
                dict(b_scales=s.double()), dict(b_scales=s.half()), dict(bias=s),
                dict(bias=s.half()[:2]), dict(out=torch.empty(4, 5, device="cuda")),
                dict(out=torch.empty(4, 4, device="cuda").t()[:, ::2])):
        kw = dict(a=q, a_scales=s, b=q, b_scales=s) | bad
        with pytest.raises(ValueError):
            armx.matmul_int8(**kw)
    with pytest.raises(TypeError):
        armx.matmul_int8(q, s, q, s, dtype=torch.float64)
    with pytest.raises(TypeError):
        armx.matmul_int8(q, s, q.float(), s)
    with pytest.raises(armx.ArmxError) as e:       # rows that start off 16 bytes
        armx.matmul_int8(torch.zeros(4, 40, dtype=torch.int8, device="cuda"), s,
                         torch.zeros(4, 40, dtype=torch.int8, device="cuda"), s)
    assert e.value.name == "ARMX_ERR_ALIGN"
    # a last row that ends inside its last 16 codes
    short = torch.zeros(3 * 48 + 40, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError, match="multiple of 16"):
        v = torch.as_strided(short, (4, 40), (48, 1))
        armx.matmul_int8(v, s, v, s)


def test_operands_past_32_bits():
    # 300k rows of 16384 codes: 4.9 GB; only the first and last rows differ from zero
    rows, k = 300_000, 16384
    b = torch.zeros(rows, k, dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(4)
    ends = make_codes(rng, 40, k, 0, "cuda")
    b[:20], b[-20:] = ends[:20], ends[20:]
    a = make_codes(rng, 3, k, 0, "cuda")
    sa, sb = scales(rng, 3), torch.ones(rows, device="cuda")
    got = armx.matmul_int8(a, sa, b, sb, dtype=torch.float32)
    want = armx.matmul_int8(a, sa, ends, sb[:40], dtype=torch.float32)
    assert torch.equal(got[:, :20], want[:, :20]) and torch.equal(got[:, -20:], want[:, 20:])
    assert not got[:, 20:-20].any()
    # and as the left operand, whose output passes 2^31 bytes
    got = armx.matmul_int8(b, sb, make_codes(rng, 4096, k, 0, "cuda"),
                           torch.ones(4096, device="cuda"), dtype=torch.float16)
    assert not got[20:-20].any() and got[:20].any() and got[-20:].any()
