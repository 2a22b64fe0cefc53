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


def every_output(rows=6, cols=40):
    """Each call with every output that it takes, as (call, outputs, inputs)."""
    rng = np.random.default_rng(1)
    x, r, dy, o, s, d = (make(rng, rows, cols, torch.float16, device="cuda") for _ in range(6))
    w = torch.ones(cols, dtype=torch.float16, device="cuda")
    inv, sc, sc2, sa = (torch.ones(rows, device="cuda") for _ in range(4))
    q, q2 = (torch.zeros(rows, 48, dtype=torch.int8, device="cuda")[:, :cols] for _ in range(2))
    dw, y = torch.zeros(cols, device="cuda"), torch.zeros(rows, rows, device="cuda")
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    big = make(rng, 2000, cols, torch.float16, device="cuda")
    ones = torch.ones(2000, device="cuda")
    return [
        (lambda: armx.rms_norm_rows(x, w, residual=r, out=o, sum_out=s), (o, s), (x, r, w)),
        (lambda: armx.rms_norm_rows_int8(x, w, residual=r, out=q, scales=sc, sum_out=s),
         (q, sc, s), (x, r, w)),
        (lambda: armx.quantize_rows_int8(x, out=q2, scales=sc2), (q2, sc2), (x,)),
        (lambda: armx.rms_norm_rows_backward(dy, x, w, inv, dsum=r, out=d, dweight=dw), (d, dw),
         (dy, x, w, inv, r)),
        (lambda: armx.rms_norm_rows_backward(big, big, w, ones, dweight=dw, workspace=ws), (dw, ws),
         (big, w, ones)),
        (lambda: armx.matmul_int8(q, sa, q2, sa, out=y), (y,), (q, q2, sa)),
    ]


def test_outputs_count_as_written():
    for call, outs, ins in every_output():
        was = [t._version for t in outs + ins]
        call()
        now = [t._version for t in outs + ins]
        n = len(outs)
        assert all(b > a for a, b in zip(was[:n], now[:n])) and was[n:] == now[n:]
    # a result made by the call is new, and a refused call writes nothing
    x = torch.ones(4, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    assert armx.rms_norm_rows(x, w).out._version == 0
    was = x._version
    with pytest.raises(armx.ArmxError):
        armx.rms_norm_rows(x, w, out=x, eps=-1.0)
    assert x._version == was


def test_a_backward_pass_notices_what_was_written_over():
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for write in (lambda t: armx.rms_norm_rows(t, w, out=t),
                  lambda t: armx.rms_norm_rows(t, w, residual=w.expand(4, 64).contiguous(), sum_out=t),
                  lambda t: armx.rms_norm_rows_backward(t, t, w, torch.ones(4, device="cuda"), out=t)):
        leaf = torch.ones(4, 64, dtype=torch.float16, device="cuda", requires_grad=True)
        y = torch.sigmoid(leaf)             # saves its result
        loss = y.sum()
        write(y.detach())
        with pytest.raises(RuntimeError, match="inplace|in-place"):
            loss.backward()


def test_outputs_made_in_inference_mode():
    with torch.inference_mode():
        calls = every_output()
        for call, _, _ in calls:
            call()
    for call, _, _ in calls:
        call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("m,n", [(1, 5), (2, 1), (7, 60), (33, 1003), (130, 4100)])
def test_a_product_feeds_the_next_operator(m, n, dtype):
    rng = np.random.default_rng([m, n])
    a, b = (armx.quantize_rows_int8(make(rng, rows, 200, dtype, device="cuda")) for rows in (m, n))
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).to(dtype).cuda()
    y = armx.matmul_int8(*a, *b, dtype=dtype)
    assert y.shape == (m, n)
    wide = make(rng, m, n, dtype, device="cuda")      # the same values in a matrix of its own
    wide.copy_(y)
    flat = torch.empty(m, n, dtype=dtype, device="cuda")
    assert torch.equal(armx.matmul_int8(*a, *b, out=flat), y)
    r = make(rng, m, n, dtype, device="cuda")
    for f in (lambda t: armx.rms_norm_rows(t, w, residual=r),
              lambda t: armx.rms_norm_rows(r, w, residual=t),
              lambda t: armx.rms_norm_rows_int8(t, w, residual=r), armx.quantize_rows_int8,
              lambda t: armx.rms_norm_rows_backward(t, r, w, torch.ones(m, device="cuda"), dsum=t)):
        for got, want in zip(f(y), f(wide)):
            assert (got is None and want is None) or torch.equal(got, want)
    assert armx.matmul_int8(*a, *b, dtype=torch.float32).is_contiguous()


@pytest.mark.parametrize("cols", [1, 13, 1003, 5001])
def test_results_of_odd_width(cols):
    # their rows' pitch, the memory behind their last row, and what PyTorch makes of them
    rng = np.random.default_rng(cols)
    x = make(rng, 3, cols, torch.float16, device="cuda")
    w = torch.ones(cols, dtype=torch.float16, device="cuda")
    n = armx.rms_norm_rows(x, w, residual=x, keep_inv_rms=True)
    q = armx.rms_norm_rows_int8(x, w, residual=x)
    g = armx.rms_norm_rows_backward(x, n.sum, w, n.inv_rms)
    for t, multiple in ((n.out, 8), (n.sum, 8), (q.sum, 8), (g.dx, 8), (q.codes, 16)):
        pitch = t.stride(0)
        assert t.shape == (3, cols) and t.stride(1) == 1 and t.storage_offset() == 0
        assert pitch % multiple == 0 and pitch >= cols and not t.is_contiguous()
        assert t.untyped_storage().nbytes() >= 3 * pitch * t.element_size()
        assert t.numel() == 3 * cols and t._base is None
        flat = torch.cat([t[i] for i in range(3)])
        assert torch.equal(t.contiguous().view(-1), flat) and torch.equal(t.clone(), t)
        assert torch.equal(t.cpu().reshape(-1), flat.cpu())
