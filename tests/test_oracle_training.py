"""The oracle of layer norm, dropout and the cross entropy: published known answers of
the generator, and its gradients against differences."""
import numpy as np

from oracle import training


def test_philox_known_answers():
    # the known answers that its authors publish for ten rounds
    for counter, key, want in [
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])]:
        assert [int(v) for v in training.philox(counter, key)] == want


def test_kept_share_and_independence():
    n = 512 * 1001
    for p in (0.0, 0.1, 0.5, 0.9, 1.0):
        keep, scale = training.kept(p, 7, 3, 512, 1001)
        # six standard deviations of a count of n draws
        assert abs(keep.mean() - (1 - p)) <= 6 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -16
        # t is off 65536 p by at most a half, so 1 - t / 65536 is off 1 - p by at most 2^-17,
        # and the scale's product with 1 - p off 1 by that over 1 - p (1.01: higher orders,
        # and the scale's own rounding)
        assert p == 1.0 or abs(scale * (1 - p) - 1) <= 1.01 * 2.0 ** -17 / (1 - p)
    a, _ = training.kept(0.5, 7, 3, 64, 1000)
    for other in (dict(seed=8, offset=3), dict(seed=7, offset=4), dict(seed=7, offset=3 + (1 << 32))):
        b, _ = training.kept(0.5, rows=64, cols=1000, **other)
        assert abs((a == b).mean() - 0.5) < 6 * 0.5 / 64000 ** 0.5
    part, _ = training.kept(0.5, 7, 3, 10, 1000, first_row=50)
    assert np.array_equal(part, a[50:60])


def differences(f, x, d=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = d
        g[i] = (f(x + e) - f(x - e)) / (2 * d)
    return g


def test_gradients_against_differences():
    rng = np.random.default_rng(3)
    h, w, b = rng.standard_normal((4, 9)) + 3, rng.standard_normal(9), rng.standard_normal(9)
    dy = rng.standard_normal((4, 9))
    _, mean, inv = training.layer_norm(h, w, b, 1e-3)
    dh, dw, db, *_ = training.layer_norm_backward(dy, h, w, mean, inv)

    def loss(h=h, w=w, b=b):
        return (training.layer_norm(h, w, b, 1e-3)[0] * dy).sum()
    assert np.allclose(dh, differences(lambda v: loss(h=v), h), atol=1e-7)
    assert np.allclose(dw, differences(lambda v: loss(w=v), w), atol=1e-7)
    assert np.allclose(db, differences(lambda v: loss(b=v), b), atol=1e-7)

    x, w = rng.standard_normal((5, 4)), rng.standard_normal((7, 4))
    t, g = np.array([0, 6, -100, 3, 3]), rng.standard_normal(5)
    loss, lse, _ = training.cross_entropy(x, w, t)
    assert loss[2] == 0
    dx, dw, _ = training.cross_entropy_backward(g, x, w, t, lse)
    assert np.allclose(dx, differences(lambda v: (training.cross_entropy(v, w, t)[0] * g).sum(), x),
                       atol=1e-7)
    assert np.allclose(dw, differences(lambda v: (training.cross_entropy(x, v, t)[0] * g).sum(), w),
                       atol=1e-7)
