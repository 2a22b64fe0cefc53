"""matmul_int8 through every tile, each at the lengths that end its pipeline in a
different way (fewer steps than buffers, as many, more; a last step of one code or
a whole one) and with ragged edges on both sides, bit for bit; the shapes choose
the tiles on a device of 256 compute units, and are right on any."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _layer import make_codes
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
CASES = [(m, n, k) for shapes in SHAPES.values() for m, n, ks in shapes for k in ks]


@pytest.mark.parametrize("m,n,k", CASES)
def test_every_tile(m, n, k):
    rng = np.random.default_rng([m, n, k])
    a, b = make_codes(rng, m, k, 1, "cuda"), make_codes(rng, n, k, 0, "cuda")
    sa, sb = scales(rng, m), scales(rng, n)
    bias = torch.from_numpy(rng.standard_normal(n)).bfloat16().cuda()
    got = armx.matmul_int8(a, sa, b, sb, bias=bias, dtype=torch.bfloat16)
    assert same(got, expected(a, sa, b, sb, bias, torch.bfloat16))
    # the same rows through other tiles
    for lo, hi in ((0, 1), (m // 2, m // 2 + 3), (m - 5, m)):
        part = armx.matmul_int8(a[lo:hi], sa[lo:hi], b, sb, bias=bias, dtype=torch.bfloat16)
        assert torch.equal(part, got[lo:hi])


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
