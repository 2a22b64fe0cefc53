"""Dropout, layer norm and the cross entropy as a training step uses them: a block's
output dropped out and added to the stream, the norm, the loss over a vocabulary, and
all the way back; eagerly, captured and replayed with a step that the graph advances,
and on several streams."""
import numpy as np
import pytest
import torch

import arithmetic_reduction_matrix_amd as armx
from oracle import training

from _layer import HALF, U, f32, f64, make
from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


V, D = 1500, 200


class Head:
    """The last block's end and the loss: h = r + dropout(x); y = norm(h) w + b; the loss of
    y against `out`, as a mean over the rows that have a target."""

    def __init__(self, dtype=torch.bfloat16):
        rng = np.random.default_rng(5)
        self.dtype = dtype
        self.w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).to(dtype).cuda()
        self.b = torch.from_numpy(0.2 * rng.standard_normal(D)).to(dtype).cuda()
        self.out = make(rng, V, D, dtype, D ** -0.5, device="cuda")
        self.step = torch.zeros(1, dtype=torch.long, device="cuda")

    def __call__(self, x, r, t):
        drop = armx.Dropout(0.1, 1234, 1 << 32, step=self.step)
        n = armx.layer_norm_rows(x, self.w, self.b, residual=r, dropout=drop, keep_stats=True)
        loss, lse = armx.cross_entropy_rows(n.out, self.out, t)
        live = (t != -100).float()
        dloss = live / live.sum()
        g = armx.cross_entropy_rows_backward(dloss, n.out, self.out, t, lse)
        back = armx.layer_norm_rows_backward(g.dx, n.sum, self.w, n.mean, n.inv_std, dropout=drop)
        return ((loss * dloss).sum(), loss, lse, n.out, n.sum, g.dx, g.dweight, back.dx,
                back.dresidual, back.dweight, back.dbias)


def inputs(rng, rows, dtype=torch.bfloat16):
    x, r = (make(rng, rows, D, dtype, device="cuda") for _ in range(2))
    t = torch.from_numpy(rng.integers(0, V, rows)).cuda()
    t[::5] = -100
    t[0] = 7
    return x, r, t


@pytest.mark.parametrize("rows", [1, 6, 70, 300])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_step_against_64_bits(rows, dtype):
    rng = np.random.default_rng(rows)
    head = Head(dtype)
    head.step.fill_(41)
    x, r, t = inputs(rng, rows, dtype)
    mean_loss, loss, lse, y, h, dy, dout, dx, dr, dw, db = head(x, r, t)
    keep, scale = training.kept(0.1, 1234, (1 << 32) + 41, rows, D)
    assert np.array_equal(f32(h), f32(torch.from_numpy(training.dropout(f32(x), keep, scale, f32(r))).to(dtype)))
    # the whole in 64 bits, without any rounding between
    want_y, mean, inv = training.layer_norm(f64(h), f64(head.w), f64(head.b), 1e-5)
    tn = t.cpu().numpy()
    want_loss, want_lse, z = training.cross_entropy(want_y, f64(head.out), tn)
    half = HALF[dtype]
    # y is half a step off, a logit that times the magnitudes behind it (and the sums'
    # and exponentials' roundings, below 2^-16 together), a loss at most two such
    e_y = half * np.abs(want_y) * 1.01 + 2.0 ** -18
    e_z = (e_y @ np.abs(f64(head.out)).T).max(1) + 2.0 ** -16 * (1 + np.abs(z).max(1))
    assert np.all(np.abs(f64(lse) - want_lse) <= e_z)
    assert np.all(np.abs(f64(loss) - want_loss) <= 2 * e_z)
    live = tn != -100
    g = live / live.sum()
    assert abs(float(mean_loss) - (want_loss * g).sum()) <= (2 * e_z * g).sum() + 2.0 ** -20 * rows
    # and back: dz's relative error is e_z and its own rounding; the vocabulary's gradient
    # and the norm's from that (to first order, half as much again for the rest)
    want_dy, want_dout, dz = training.cross_entropy_backward(g, want_y, f64(head.out), tn, want_lse)
    p = np.abs(dz)
    e_dz = p * (half + 2 * e_z[:, None]) + (g * 2 * e_z)[:, None] * np.exp(z - want_lse[:, None])
    tiny = 2.0 ** -24   # binary16's smallest step
    e_dy = (e_dz @ np.abs(f64(head.out)) + half * np.abs(want_dy)) * 1.5 + tiny
    assert np.all(np.abs(f64(dy) - want_dy) <= e_dy)
    e_dout = (e_dz.T @ np.abs(want_y) + p.T @ e_y + half * np.abs(want_dout)) * 1.5 + tiny
    assert np.all(np.abs(f64(dout) - want_dout) <= e_dout)
    w = np.abs(f64(head.w))
    dh, want_dw, want_db, (ag, mg, mgn, n, i), *_ = training.layer_norm_backward(
        want_dy, f64(h), f64(head.w), mean, inv)
    eg = e_dy * w
    e_dh = (i * (eg + eg.mean(1, keepdims=True) + n * (eg * n).mean(1, keepdims=True))
            + half * np.abs(dh)) * 1.5 + 2.0 ** -18 * i * (ag + mg + n * mgn) + tiny
    assert np.all(np.abs(f64(dr) - dh) <= e_dh)
    assert np.all(np.abs(f64(dx) - np.where(keep, dh * float(scale), 0)) <= e_dh * 1.2)
    assert np.all(np.abs(f64(db) - want_db) <= e_dy.sum(0) + 2 * U * rows * np.abs(want_dy).sum(0))
    assert np.all(np.abs(f64(dw) - want_dw) <= (e_dy * (n + 2.0 ** -16)).sum(0)
                  + 2.0 ** -16 * np.abs(want_dy * n).sum(0))


def test_captured_and_replayed_with_a_step_of_its_own():
    rng = np.random.default_rng(3)
    head, eager = Head(), Head()
    x, r, t = inputs(rng, 150)
    head(x, r, t)   # what is built on the first call
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        head(x, r, t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = head(x, r, t)
        head.step.add_(1)   # behind the backward pass, which reads it too
    assert int(head.step) == 0
    seen = []
    for replay in range(5):
        nx, nr, nt = inputs(rng, 150)
        for a, b in zip((x, r, t), (nx, nr, nt)):
            a.copy_(b)
        eager.step.fill_(replay)
        want = eager(nx, nr, nt)
        graph.replay()
        torch.cuda.synchronize()
        assert int(head.step) == replay + 1
        # the mean's own sum is torch's
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:])), replay
        seen.append((got[7] == 0).cpu())
        nx.zero_()
        torch.cuda.synchronize()
    # another mask each time
    assert all(not torch.equal(a, b) for a, b in zip(seen, seen[1:]))


def test_two_graphs_and_eager_calls_share_nothing():
    rng = np.random.default_rng(4)
    head = Head()
    sets = [inputs(rng, n) for n in (40, 200)]
    want = [head(*s) for s in sets]
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(head(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        mixed = [head(*s) for s in sets]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b, c in zip(want, outs, mixed):
            assert all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))
            assert all(torch.equal(p, q) for p, q in zip(a[1:], c[1:]))


def test_streams_of_their_own():
    rng = np.random.default_rng(6)
    head = Head()
    sets = [inputs(rng, n) for n in (3, 130, 260)]
    want = [head(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, args in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(head(*args))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))


def test_events_are_stamped():
    rng = np.random.default_rng(7)
    x, r, t = inputs(rng, 300)
    head = Head()
    d = armx.Dropout(0.1, 1)
    n = armx.layer_norm_rows(x, head.w, residual=r, keep_stats=True)
    lse = armx.cross_entropy_rows(x, head.out, t).lse
    g = torch.ones(300, device="cuda")
    big = make(rng, 2000, D, torch.bfloat16, device="cuda")
    bn = armx.layer_norm_rows(big, head.w, keep_stats=True)
    for call in (lambda **e: armx.dropout_rows(x, d, **e),
                 lambda **e: armx.layer_norm_rows(x, head.w, dropout=d, **e),
                 lambda **e: armx.layer_norm_rows_backward(x, n.sum, head.w, n.mean, n.inv_std, **e),
                 lambda **e: armx.layer_norm_rows_backward(big, big, head.w, bn.mean, bn.inv_std, **e),
                 lambda **e: armx.cross_entropy_rows(x, head.out, t, **e),
                 lambda **e: armx.cross_entropy_rows_backward(g, x, head.out, t, lse, **e),
                 lambda **e: armx.cross_entropy_rows_backward(g, x, head.out, t, lse, need_dx=False, **e)):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        call(start_event=a, stop_event=b)
        torch.cuda.synchronize()
        assert 0 < a.elapsed_time(b) < 1000
