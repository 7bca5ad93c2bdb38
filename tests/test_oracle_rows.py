"""Pins of the fp64 oracle of the gated linear recurrence and the row norms
(``oracle/rows.py``): explicit products, closed forms, split invariance and
finite differences (CPU only)."""
import numpy as np
import pytest

from oracle import rows


def draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


FORMS = [(gate, tied) for gate in ("value", "logit") for tied in (False, True)]


def make(seed, B, T, D, gate):
    g = draw(seed + 1, B, T, D)
    return draw(seed, B, T, D), (g if gate == "logit" else 1.0 / (1.0 + np.exp(-g))), draw(seed + 2, B, D)


@pytest.mark.parametrize("gate,tied", FORMS)
def test_scan_is_the_sum_of_decayed_inputs(gate, tied):
    x, g, h0 = make(1, 2, 9, 3, gate)
    a = 1.0 / (1.0 + np.exp(-g)) if gate == "logit" else g
    u = (1.0 - a) * x if tied else x
    h, last = rows.scan_fwd(x, g, h0, gate, tied)
    for t in range(9):
        want = np.prod(a[:, :t + 1], axis=1) * h0
        for i in range(t + 1):
            want = want + np.prod(a[:, i + 1:t + 1], axis=1) * u[:, i]
        assert np.allclose(h[:, t], want, rtol=1e-13, atol=1e-14)
    assert np.array_equal(last, h[:, -1])


def test_scan_closed_forms():
    T = 7
    one = np.ones((1, T, 2))
    h, _ = rows.scan_fwd(one, 0.5 * one)                       # geometric sum
    assert np.allclose(h[0, :, 0], 2.0 - 0.5 ** np.arange(T), rtol=1e-15)
    h, last = rows.scan_fwd(one, one, np.full((1, 2), 3.0))     # a = 1 counts
    assert np.array_equal(h[0, :, 1], 3.0 + np.arange(1, T + 1))
    h, _ = rows.scan_fwd(5 * one, 0.3 * one, np.full((1, 2), 5.0), tied=True)
    assert np.allclose(h, 5.0, rtol=1e-15)                      # a tied input's fixed point
    h, last = rows.scan_fwd(one[:, :0], one[:, :0], np.full((1, 2), 4.0))
    assert h.shape == (1, 0, 2) and np.array_equal(last, np.full((1, 2), 4.0))
    h, _ = rows.scan_fwd(one, np.full((1, T, 2), 1000.0), gate="logit", tied=True)
    assert np.all(h == 0.0)                                     # an open gate takes no tied input
    h, _ = rows.scan_fwd(one, np.full((1, T, 2), -1000.0), gate="logit", tied=True)
    assert np.all(h == 1.0)


@pytest.mark.parametrize("gate,tied", FORMS)
def test_scan_split_invariance(gate, tied):
    x, g, h0 = make(4, 2, 11, 3, gate)
    h, last = rows.scan_fwd(x, g, h0, gate, tied)
    for cut in (0, 1, 6, 11):
        h1, mid = rows.scan_fwd(x[:, :cut], g[:, :cut], h0, gate, tied)
        h2, end = rows.scan_fwd(x[:, cut:], g[:, cut:], mid, gate, tied)
        assert np.array_equal(np.concatenate([h1, h2], 1), h) and np.array_equal(end, last)


@pytest.mark.parametrize("gate,tied", FORMS)
def test_scan_gradients_are_differences(gate, tied):
    x, g, h0 = make(7, 2, 6, 3, gate)
    dh, dl = draw(20, 2, 6, 3), draw(21, 2, 3)

    def loss(x, g, h0):
        h, last = rows.scan_fwd(x, g, h0, gate, tied)
        return (h * dh).sum() + (last * dl).sum()

    h, _ = rows.scan_fwd(x, g, h0, gate, tied)
    got = rows.scan_bwd(g, h, dh, x, h0, dl, gate, tied)
    inputs, e = [x, g, h0], 1e-6
    for k in range(3):
        it = np.nditer(inputs[k], flags=["multi_index"])
        for _ in it:
            i = it.multi_index
            p, m = [a.copy() for a in inputs], [a.copy() for a in inputs]
            p[k][i] += e
            m[k][i] -= e
            assert abs((loss(*p) - loss(*m)) / (2 * e) - got[k][i]) <= 1e-7 * (1 + abs(got[k][i]))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_rows(kind):
    x, w, b = draw(30, 5, 8), draw(31, 8), draw(32, 8)
    y, mean, rstd = rows.norm_fwd(x, kind=kind, eps=1e-300)
    assert np.allclose((y * y).mean(1), 1.0, rtol=1e-14)
    if kind == "layer":
        assert np.allclose(y.mean(1), 0.0, atol=1e-15)
        assert np.allclose(rows.norm_fwd(x + 7.0, kind=kind, eps=1e-300)[0], y, rtol=1e-12, atol=1e-13)
    assert np.allclose(rows.norm_fwd(-3.0 * x, kind=kind, eps=1e-300)[0], -y, rtol=1e-13)
    assert np.allclose(rows.norm_fwd(x, w, b, kind, 1e-300)[0], y * w + b, rtol=1e-15)
    c = rows.norm_fwd(np.full((2, 8), 3.0), kind=kind, eps=0.25)
    if kind == "layer":                                         # a constant row has no deviation
        assert np.array_equal(c[0], np.zeros((2, 8))) and np.array_equal(c[2], np.full(2, 2.0))
    else:
        assert np.allclose(c[0], 3.0 / np.sqrt(9.25), rtol=1e-15)
    assert np.allclose(rows.norm_fwd(np.array([[3.0, 4.0, 0.0, 0.0]]), kind="rms", eps=1e-300)[0],
                       [[1.2, 1.6, 0.0, 0.0]], rtol=1e-15)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_are_differences(kind):
    x, w, b, dy = draw(40, 3, 5), draw(41, 5), draw(42, 5), draw(43, 3, 5)

    def loss(x, w, b):
        return (rows.norm_fwd(x, w, b, kind, 0.1)[0] * dy).sum()

    _, mean, rstd = rows.norm_fwd(x, w, b, kind, 0.1)
    got = rows.norm_bwd(dy, x, rstd, mean, w, kind)
    inputs, e = [x, w, b], 1e-6
    for k in range(3):
        it = np.nditer(inputs[k], flags=["multi_index"])
        for _ in it:
            i = it.multi_index
            p, m = [a.copy() for a in inputs], [a.copy() for a in inputs]
            p[k][i] += e
            m[k][i] -= e
            assert abs((loss(*p) - loss(*m)) / (2 * e) - got[k][i]) <= 1e-7 * (1 + abs(got[k][i]))
