"""The layer operators at the ends of what their documentation allows."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx

from _layer import TYPES, f64, ids, make
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [24, 600, 3000, 20000, 40000])
def test_codes_of_rows_of_zeros_without_eps(cols, dtype):
    # 1 / rms is an infinity there; codes and scale are 0, and so is their product
    rng = np.random.default_rng(cols)
    x = make(rng, 5, cols, dtype)
    x[0], x[3] = 0.0, -0.0
    x = x.cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(cols)).to(dtype).cuda()
    minus = make(rng, 5, cols, dtype, device="cuda")
    minus.copy_(-x)
    minus[2] = 0.0
    for residual, zeros in ((None, [0, 3]), (minus, [0, 1, 3, 4])):
        n = armx.rms_norm_rows_int8(x, w, residual=residual, eps=0.0)
        others = [r for r in range(5) if r not in zeros]
        assert not n.codes[zeros].any() and not n.scales[zeros].any()
        assert np.all(f64(n.scales)[others] > 0) and np.isfinite(f64(n.scales)).all()
        assert n.codes[others].abs().amax(1).eq(127).all()
        y = armx.matmul_int8(n.codes, n.scales, n.codes, n.scales, dtype=torch.float32)
        assert not y[zeros].any() and not y[:, zeros].any() and torch.isfinite(y).all()
