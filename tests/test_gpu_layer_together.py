"""The layer operators as a model uses them: norm with the residual into codes,
the product with quantised weights, a second norm, and the training form's
forward and backward; eagerly, captured and replayed, and on several streams."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import layer

from _layer import HALF, U, f32, f64, make
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


D, F = 1000, 2300


class Block:
    """Two quantised projections around norms: h = x + r; z = norm(h) A; then the
    codes of z; y = z B, and the next norm of h + y."""

    def __init__(self, dtype=torch.bfloat16):
        rng = np.random.default_rng(11)
        self.dtype = dtype
        self.w1, self.w2 = (torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).to(dtype).cuda()
                            for _ in range(2))
        self.a = make(rng, F, D, dtype, D ** -0.5, device="cuda")
        self.b = make(rng, D, F, dtype, F ** -0.5, device="cuda")
        self.bias = torch.from_numpy(rng.standard_normal(F)).to(dtype).cuda()
        self.aq, self.bq = armx.quantize_rows_int8(self.a), armx.quantize_rows_int8(self.b)

    def __call__(self, x, r):
        n = armx.rms_norm_rows_int8(x, self.w1, residual=r)
        # the product's rows are read by the quantiser: whole 16-byte rows
        z = torch.empty(x.shape[0], -(-F // 8) * 8, dtype=self.dtype, device=x.device)[:, :F]
        armx.matmul_int8(n.codes, n.scales, self.aq.codes, self.aq.scales, bias=self.bias, out=z)
        q = armx.quantize_rows_int8(z)
        y = armx.matmul_int8(q.codes, q.scales, self.bq.codes, self.bq.scales, dtype=self.dtype)
        last = armx.rms_norm_rows(y, self.w2, residual=n.sum)
        return last.out, last.sum, z, n


def outputs(b, x, r):
    out, s, z, n = b(x, r)
    return out, s, z, n.codes, n.scales, n.sum


@pytest.mark.parametrize("rows", [1, 5, 70, 300])
def test_block_against_64_bits(rows):
    rng = np.random.default_rng(rows)
    blk = Block()
    x, r = (make(rng, rows, D, torch.bfloat16, device="cuda") for _ in range(2))
    out, s, z, n = blk(x, r)
    # each stage from the stage before it, in 64 bits
    h = f64((x.float() + r.float()).bfloat16())
    assert np.array_equal(f64(n.sum), h)
    q, top = layer.codes(np.float32(h) * f32(blk.w1))
    assert np.array_equal(n.codes.cpu().numpy(), q)
    want = layer.product(q, blk.aq.codes.cpu().numpy()) * f64(n.scales)[:, None] * f64(blk.aq.scales)
    big = np.abs(want) + np.abs(f64(blk.bias))
    want = want + f64(blk.bias)
    assert np.all(np.abs(f64(z) - want) <= HALF[torch.bfloat16] * np.abs(want) * 1.01 + 5 * U * big)
    # and the whole against unquantised 64 bits: a code is off by half a step of
    # its row's 127th, so a product of k codes by at most the sum of both sides' halves
    norm, _ = layer.rms_norm(h, f64(blk.w1), 1e-6)
    full = norm @ f64(blk.a).T + f64(blk.bias)
    sa, sb = f64(n.scales)[:, None], f64(blk.aq.scales)[None, :]
    bound = 0.5 * (sa * np.abs(f64(blk.a)).sum(1)[None, :] + np.abs(norm).sum(1)[:, None] * sb
                   + 0.5 * D * sa * sb)
    assert np.all(np.abs(f64(z) - full) <= 1.01 * bound + HALF[torch.bfloat16] * 1.01 * (np.abs(full) + bound))
    # rows of a batch are rows alone
    o1, s1, *_ = blk(x[rows // 2:rows // 2 + 1], r[rows // 2:rows // 2 + 1])
    assert torch.equal(o1[0], out[rows // 2]) and torch.equal(s1[0], s[rows // 2])


def test_training_step_through_two_norms():
    # forward: s1 = x + r, y1 = norm(s1); s2 = s1 + y1, y2 = norm(s2); loss = <y2, dy>
    rng = np.random.default_rng(3)
    rows, cols = 40, 1200
    t = torch.float16
    x, r, dy = (make(rng, rows, cols, t, device="cuda") for _ in range(3))
    w1, w2 = (torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).to(t).cuda() for _ in range(2))
    n1 = armx.rms_norm_rows(x, w1, residual=r, keep_inv_rms=True)
    n2 = armx.rms_norm_rows(n1.out, w2, residual=n1.sum, keep_inv_rms=True)
    g2 = armx.rms_norm_rows_backward(dy, n2.sum, w2, n2.inv_rms)
    g1 = armx.rms_norm_rows_backward(g2.dx, n1.sum, w1, n1.inv_rms, dsum=g2.dx)
    # float64 autograd over the same graph on the CPU
    leaves = [v.cpu().double().requires_grad_() for v in (x, r, w1, w2)]
    X, R, W1, W2 = leaves

    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * w
    s1 = X + R
    s2 = s1 + norm(s1, W1)
    (norm(s2, W2) * dy.cpu().double()).sum().backward()
    # roundings to 16 bits on the way: s1, y1, s2 and the two dx, each half a
    # step of values of the rows' size; eight steps bound the five and what
    # they move (the norm's derivative has norm at most max w / rms, near 1)
    for got, want in ((g1.dx, X.grad), (g1.dx, R.grad), (g1.dweight, W1.grad), (g2.dweight, W2.grad)):
        want = want.numpy()
        err = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert err <= 16 * HALF[t], err


def test_captured_and_replayed():
    blk = Block()
    rng = np.random.default_rng(5)
    rows = 33
    pool = [[make(rng, rows, D, torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(4)]
    x, r = (t.clone() for t in pool[0])
    w = blk.w1
    big = make(rng, 3000, D, torch.bfloat16, device="cuda")    # a backward with a workspace

    def calls():
        out = outputs(blk, x, r)
        n = armx.rms_norm_rows(big, w, keep_inv_rms=True)
        g = armx.rms_norm_rows_backward(big, big, w, n.inv_rms)
        return (*out, g.dx, g.dweight)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                # two graphs of the same calls, alive together
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = calls()
        graphs.append((g, got))
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(4):
        x.copy_(pool[rep][0])
        r.copy_(pool[rep][1])
        big.mul_(-1.0)
        torch.cuda.synchronize()
        for s, (g, _) in zip(streams, graphs):      # replayed at the same time
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = calls()
        torch.cuda.synchronize()
        for _, got in graphs:
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), (rep, i)


def test_streams_at_the_same_time():
    blk = Block()
    rng = np.random.default_rng(6)
    ins = [[make(rng, 50 + 60 * i, D, torch.bfloat16, device="cuda") for _ in range(2)] for i in range(4)]
    want = [outputs(blk, *v) for v in ins]
    grads = []
    for x, _ in ins:
        n = armx.rms_norm_rows(x, blk.w1, keep_inv_rms=True)
        grads.append(armx.rms_norm_rows_backward(x, x, blk.w1, n.inv_rms))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None] * 4
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                o = outputs(blk, *ins[i])
                n = armx.rms_norm_rows(ins[i][0], blk.w1, keep_inv_rms=True)
                got[i] = (o, armx.rms_norm_rows_backward(ins[i][0], ins[i][0], blk.w1, n.inv_rms))
    torch.cuda.synchronize()
    for i in range(4):
        for a, b in zip((*got[i][0], *got[i][1]), (*want[i], *grads[i])):
            assert torch.equal(a, b), i


def test_events_and_log(capfd):
    x = torch.ones(4, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    n = armx.rms_norm_rows(x, w, keep_inv_rms=True, start_event=start, stop_event=stop)
    torch.cuda.synchronize()
    assert 0 <= start.elapsed_time(stop) < 1000
    big = torch.ones(5000, 64, dtype=torch.float16, device="cuda")
    inv = armx.rms_norm_rows(big, w, keep_inv_rms=True).inv_rms
    armx.rms_norm_rows_backward(big, big, w, inv, start_event=start, stop_event=stop)
    torch.cuda.synchronize()
    assert 0 <= start.elapsed_time(stop) < 1000
    q = armx.quantize_rows_int8(x, start_event=start, stop_event=stop)
    armx.matmul_int8(q.codes, q.scales, q.codes, q.scales, start_event=start, stop_event=stop)
    torch.cuda.synchronize()
    assert 0 <= start.elapsed_time(stop) < 1000 and n.inv_rms.numel() == 4
    assert "armx:" not in capfd.readouterr().err
