"""Pins of the float64 reference of the training side: gradients against
differences, the codecs against enumeration, the stochastic rounding's mean."""

import numpy as np
import pytest

from oracle import train as T

RNG = np.random.default_rng


def _layer(x, w1, w2, start, rows, weight):
    pre, _ = T.grouped_forward(x, w1, start, rows)
    s = np.concatenate([i for _, i in T.spans(start, rows)])
    h = np.zeros((x.shape[0], w1.shape[1] // 2))
    h[s] = T.swiglu(pre[s], weight[s])
    y, _ = T.grouped_forward(h, w2, start, rows)
    return pre, h, y, s


def test_gradients_match_differences():
    """d(sum c * y) through both products and the activation, by central differences."""
    g = RNG(1)
    E, H, I, start, rows = 3, 5, 4, [2, 0, 7], [3, 0, 2]
    x, w1, w2 = g.standard_normal((9, H)), g.standard_normal((E, 2 * I, H)), g.standard_normal((E, H, I))
    wt, c = g.uniform(0.2, 1, 9), g.standard_normal((9, H))
    pre, h, y, s = _layer(x, w1, w2, start, rows, wt)
    dy = np.zeros_like(c)
    dy[s] = c[s]
    dh, _ = T.grouped_input_gradient(dy, w2, start, rows)
    dw2, _ = T.grouped_wgrad(dy, h, start, rows)
    dpre, h2, dwt = (np.zeros((9, 2 * I)), np.zeros((9, I)), np.zeros(9))
    dpre[s], h2[s], dwt[s] = T.swiglu_backward(dh[s], pre[s], wt[s])
    np.testing.assert_allclose(h2[s], h[s], rtol=1e-14)
    dx, _ = T.grouped_input_gradient(dpre, w1, start, rows)
    dw1, _ = T.grouped_wgrad(dpre, x, start, rows)

    def loss():
        return float((c[s] * _layer(x, w1, w2, start, rows, wt)[2][s]).sum())

    for a, da in ((x, np.nan_to_num(dx)), (w1, dw1), (w2, dw2), (wt, dwt)):
        flat, dflat = a.reshape(-1), da.reshape(-1)
        for k in g.choice(flat.size, min(flat.size, 25), replace=False):
            old = flat[k]
            vals = []
            for d in (1e-5, -1e-5):
                flat[k] = old + d
                vals.append(loss())
            flat[k] = old
            # central differences: third derivatives (order 10) times 1e-10, rounding 1e-14 / 1e-5
            assert abs((vals[0] - vals[1]) / 2e-5 - dflat[k]) <= 1e-7 * (1 + abs(dflat[k]))


def _all_codes():
    return np.array([v for e in range(16) for m in range(8) if not (e == 15 and m == 7)
                     for v in [(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)]])


def test_e4m3_nearest_is_the_nearest_code():
    codes = _all_codes()
    assert codes[-1] == 448 and len(codes) == 127
    y = np.concatenate([codes, (codes[1:] + codes[:-1]) / 2, RNG(2).uniform(0, 448, 500), 2.0 ** RNG(3).uniform(-12, 8, 500)])
    q = T.e4m3_nearest(y)
    assert np.isin(q, codes).all()
    np.testing.assert_array_equal(np.abs(q - y), np.abs(codes[None] - y[:, None]).min(1))
    assert (T.e4m3_nearest(-y) == -q).all()


def test_e4m3_random_rounds_to_a_neighbour_with_the_right_mean():
    codes = _all_codes()
    u = np.arange(1 << 20, dtype=np.int64)
    for y in [1.0, 1.03, 300.7, 447.9, 2.0 ** -6 * 1.01, 2.0 ** -7 * 1.3, 2.0 ** -9 * 1.5, 448.0]:
        q = T.e4m3_random(np.full(u.size, y), u)
        lo, hi = codes[codes <= y].max(), codes[codes >= y].min()
        assert set(np.unique(q)) <= {lo, hi}
        assert abs(q.mean() - y) <= 2 * T.e4m3_spacing(np.array([y]))[0] / 2 ** 20
    assert T.e4m3_random(np.array([0.0]), np.array([5]))[0] == 0
    assert T.e4m3_random(np.array([1e-9]), np.array([0]))[0] == 2.0 ** -9


def test_hash_bits_are_spread():
    h = T.hash20(7, 0, 20000)
    assert h.min() >= 0 and h.max() < 1 << 20
    # mean of 20000 uniform values: standard deviation 2^20 / sqrt(12 * 20000)
    assert abs(h.mean() / 2 ** 20 - 0.5) < 5 / np.sqrt(12 * 20000)
    assert (T.hash20(8, 0, 50) != h[:50]).any() and (T.hash20(7, 1, 50) != h[:50]).any()
    assert (T.hash20(7, 0, 50, first=(1 << 33) + 5) != h[5:55]).any()


def test_adamw_first_step_moves_by_the_learning_rate():
    """After one step from zero states the update is lr * sign(g) (eps = 0)."""
    g = RNG(4).standard_normal(50)
    p, m, v, r, upd = T.adamw(np.ones(50), g, np.zeros(50), np.zeros(50), 1e-2, 0.9, 0.999, 0.0, 0.5, 1)
    np.testing.assert_allclose(p, 1 - 1e-2 * 0.5 - 1e-2 * np.sign(g), rtol=1e-13)
    np.testing.assert_allclose(r * r, v, rtol=1e-14)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 300])
def test_group_maxima(n):
    x = RNG(n).standard_normal(n)
    want = [np.abs(x[i:i + 128]).max() for i in range(0, n, 128)]
    np.testing.assert_array_equal(T.group_max(x), want)
    assert T.per_element(T.group_max(x), n).shape == (n,)
