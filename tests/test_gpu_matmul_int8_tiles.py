"""matmul_int8 through every tile, each at the lengths that end its pipeline in a
different way (fewer steps than buffers, as many, more; a last step of one code or
a whole one) and with ragged edges on both sides, bit for bit; rows on 128-byte lines
and off them.  The shapes choose the tiles on a device of 256 compute units, and are
right on any."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _parity import require_gpu
from test_gpu_matmul_int8 import expected, same, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# (m, n, lengths) by the tile of rows x columns that they choose
SHAPES = {
    "256x256": [(520, 16300, (97, 200)), (1100, 8150, (300, 513, 640))],
    "192x192": [(520, 16300, (300, 385, 512, 650))],
    "128x256": [(1000, 6050, (97, 200, 300, 513, 1150))],
    "192x128": [(330, 12200, (97, 200, 300, 513, 1150))],
    "128x128": [(130, 12200, (300, 430, 513, 1150, 2100))],
    "64x128": [(130, 12200, (97, 200)), (130, 6050, (700, 1153, 2048))],
    "64x64": [(5, 12200, (97, 200, 300, 430, 520, 641, 2100))],
    "64x32": [(40, 6050, (300, 430, 700, 1153, 2560))],
    "32x32": [(5, 6050, (97, 200, 430)), (1500, 66, (520, 1025, 2100, 2561))],
    "16x32": [(5, 6050, (520, 1025, 2100, 3000))],
    "16x16": [(5, 66, (97, 1000, 2100, 4097, 9000))],
}
# the same where rows do not all start on a 128-byte line
OFF_LINE_SHAPES = {
    "256x256": [(520, 16300, (97, 200)), (1100, 8150, (300, 513, 640))],
    "192x192": [(520, 16300, (300, 385, 512, 650, 1153))],
    "128x256": [(1000, 6050, (97, 200, 300, 513, 1150))],
    "192x128": [(330, 12200, (300, 400, 513, 641, 1150)), (330, 12200, (2100,))],
    "128x128": [(130, 12200, (97, 200, 300, 430, 513, 641, 1150, 2100))],
    "128x64": [(130, 6050, (430, 513, 641, 700, 1153, 2048)), (70, 12200, (400,))],
    "64x64": [(5, 12200, (430, 520, 641, 700, 2100)), (70, 6050, (400, 1153))],
    "64x32": [(40, 6050, (97, 200, 300, 430, 513, 641, 700, 1153, 2560))],
    "32x32": [(1500, 66, (97, 200, 430, 520, 1025, 2561))],
    "16x32": [(5, 6050, (97, 520, 1025, 3000))],
    "16x16": [(5, 66, (97, 1000, 2100, 4097))],
}
# in pieces of 16 codes: what the pitches of a and b are past whole lines, and where
# their first rows start
STARTS = [(1, 3, 0, 0), (5, 7, 2, 1), (2, 6, 0, 4), (4, 0, 0, 0), (0, 0, 3, 5), (0, 1, 0, 0), (3, 2, 7, 6)]


def cases(shapes):
    return [(m, n, k) for several in shapes.values() for m, n, ks in several for k in ks]


def codes_at(rng, rows, k, past, start):
    """rows x k codes at a pitch `past` pieces more than whole lines, from piece `start` on."""
    pitch = -(-k // 16)
    pitch = 16 * (pitch + (past - pitch) % 8)
    flat = torch.from_numpy(rng.integers(-128, 128, 16 * start + rows * pitch, dtype=np.int8)).cuda()
    return flat[16 * start:].view(rows, pitch)[:, :k]


def check(rng, a, b):
    m, n = a.shape[0], b.shape[0]
    sa, sb = scales(rng, m), scales(rng, n)
    bias = torch.from_numpy(rng.standard_normal(n)).bfloat16().cuda()
    got = armx.matmul_int8(a, sa, b, sb, bias=bias, dtype=torch.bfloat16)
    assert same(got, expected(a, sa, b, sb, bias, torch.bfloat16))
    # the same rows through other tiles
    for lo, hi in ((0, 1), (m // 2, m // 2 + 3), (m - 5, m)):
        part = armx.matmul_int8(a[lo:hi], sa[lo:hi], b, sb, bias=bias, dtype=torch.bfloat16)
        assert torch.equal(part, got[lo:hi])


@pytest.mark.parametrize("m,n,k", cases(SHAPES))
def test_every_tile(m, n, k):
    rng = np.random.default_rng([m, n, k])
    check(rng, codes_at(rng, m, k, 0, 0), codes_at(rng, n, k, 0, 0))


@pytest.mark.parametrize("m,n,k", cases(OFF_LINE_SHAPES))
def test_every_tile_of_rows_off_the_lines(m, n, k):
    rng = np.random.default_rng([m, n, k, 1])
    which = STARTS[(m + n + k) % len(STARTS)]
    check(rng, codes_at(rng, m, k, which[0], which[2]), codes_at(rng, n, k, which[1], which[3]))


@pytest.mark.parametrize("past_a,past_b,start_a,start_b", STARTS)
def test_every_place_past_a_line(past_a, past_b, start_a, start_b):
    rng = np.random.default_rng([past_a, past_b, start_a])
    for m, n, k in ((330, 12200, 641), (70, 6050, 400), (40, 6050, 129), (520, 16300, 144)):
        check(rng, codes_at(rng, m, k, past_a, start_a), codes_at(rng, n, k, past_b, start_b))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("start,pitch", [(1, 131), (2, 132), (3, 204)])
def test_results_that_start_anywhere(start, pitch, dtype):
    # rows of the result off 4, 8 and 16 bytes, and nothing else written
    rng = np.random.default_rng([start, pitch])
    for m in (3, 70, 200):
        a, b = codes_at(rng, m, 300, 1, 0), codes_at(rng, 130, 300, 0, 0)
        sa, sb = scales(rng, m), scales(rng, 130)
        flat = torch.full((start + m * pitch + 8,), 7.0, dtype=dtype, device="cuda")
        out = flat[start:start + m * pitch].view(m, pitch)[:, :130]
        armx.matmul_int8(a, sa, b, sb, out=out)
        assert same(out.contiguous(), expected(a, sa, b, sb, None, dtype))
        out.fill_(7.0)
        assert bool((flat == 7.0).all())


def test_codes_made_here_fit_the_product():
    # pitches of 16 codes and of whole lines; the product reads either
    rng = np.random.default_rng(0)
    for cols, pitch in ((40, 48), (511, 512), (512, 512), (600, 640), (5001, 5120)):
        wide = torch.zeros(3, -(-cols // 8) * 8, dtype=torch.float16, device="cuda")
        wide[:, :cols] = torch.from_numpy(rng.standard_normal((3, cols))).half()
        q = armx.quantize_rows_int8(wide[:, :cols])
        assert q.codes.stride() == (pitch, 1)
        got = armx.matmul_int8(q.codes, q.scales, q.codes, q.scales, dtype=torch.float32)
        want = layer.product(q.codes.cpu().numpy(), q.codes.cpu().numpy())
        want = torch.from_numpy(want).float() * (q.scales.cpu()[:, None] * q.scales.cpu()[None])
        assert torch.equal(got.cpu(), want)
