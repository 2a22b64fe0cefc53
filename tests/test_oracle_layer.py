"""The layer oracle against closed forms, Fractions and differences (CPU)."""
from fractions import Fraction

import numpy as np

from oracle import layer


def test_codes_against_fractions():
    rng = np.random.default_rng(1)
    for _ in range(300):
        n = int(rng.integers(1, 20))
        p = np.float32(rng.standard_normal(n)) * np.float32(10.0 ** rng.integers(-30, 30))
        if rng.random() < 0.3:      # exact halves: whole multiples of top / 254
            p = np.float32(rng.integers(-254, 255, n)) * np.float32(2.0 ** rng.integers(-40, 40))
            p[0] = np.float32(254 * 2.0 ** -3)
        q, top = layer.codes(p[None])
        t = max(abs(Fraction(float(v))) for v in p)
        assert Fraction(float(top[0])) == t
        for v, c in zip(p, q[0]):
            want = round(127 * Fraction(float(v)) / t) if t else 0   # half to even
            assert int(c) == want, (float(v), float(top[0]))


def test_codes_of_rows_without_an_answer():
    p = np.array([[0, 0, -0.0], [1, np.inf, 2], [np.nan, 1, 2], [-3, 3, 1.5]], np.float32)
    q, top = layer.codes(p)
    assert q.tolist() == [[0, 0, 0], [0, 0, 0], [0, 0, 0], [-127, 127, 64]]   # 63.5 to even
    assert top[0] == 0 and np.isnan(top[1]) and np.isnan(top[2]) and top[3] == 3


def test_backward_against_differences():
    rng = np.random.default_rng(2)
    h, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    ds, eps, d = rng.standard_normal((3, 7)), 1e-3, 1e-6
    _, inv = layer.rms_norm(h, w, eps)
    dx, dw, *_ = layer.rms_norm_backward(dy, h, w, inv, ds)

    def loss(h, w):
        return (layer.rms_norm(h, w, eps)[0] * dy).sum() + (h * ds).sum()
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dx[i]) < 1e-7
    for j in range(7):
        e = np.zeros_like(w)
        e[j] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_rms_norm_of_a_constant_row():
    y, inv = layer.rms_norm(np.full((1, 10), -4.0), np.arange(10), 0.0)
    assert inv[0] == 0.25 and np.array_equal(y[0], -np.arange(10.0))
