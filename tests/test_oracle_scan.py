"""Pins of the recurrence's oracle: closed forms, the compositing equation and
float64 finite differences."""
import numpy as np
import pytest

from oracle import scan as O


def _case(seed, S=4, C=6, G=3):
    rng = np.random.default_rng(seed)
    lens = np.array([5, 0, 1, 7])[:S]
    off = np.concatenate([[0], np.cumsum(lens)])
    T = int(off[-1])
    return rng, off, rng.uniform(0.2, 1.0, (T, G)), rng.normal(size=(T, C)), rng.normal(size=(S, C))


def test_constant_gate_is_a_geometric_sum():
    T = 9
    h, last, _ = O.forward(np.full((T, 1), 0.5), np.ones((T, 1)), [0, T], np.full((1, 1), 4.0))
    want = [4.0 * 0.5 ** (t + 1) + (1 - 0.5 ** (t + 1)) / 0.5 for t in range(T)]
    np.testing.assert_allclose(h[:, 0], want, rtol=1e-14)
    assert last[0, 0] == h[-1, 0]


def test_coupled_reverse_is_the_compositing_equation():
    """Back to front over samples listed front to back: sum of alpha_i c_i
    prod_{j < i} (1 - alpha_j), plus the background through all of them."""
    rng = np.random.default_rng(0)
    T, C = 12, 3
    alpha, c, bg = rng.uniform(0, 1, T), rng.uniform(0, 1, (T, C)), rng.uniform(0, 1, (1, C))
    _, last, _ = O.forward(1 - alpha[:, None], c, [0, T], bg, reverse=True, coupled=True)
    trans = np.concatenate([[1.0], np.cumprod(1 - alpha)])
    want = (alpha * trans[:-1]) @ c + trans[-1] * bg[0]
    np.testing.assert_allclose(last[0], want, rtol=1e-13)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("coupled", [False, True])
def test_gradients_match_finite_differences(reverse, coupled):
    rng, off, a, x, h0 = _case(3)
    dh, dl = rng.normal(size=x.shape), rng.normal(size=h0.shape)

    def loss(a_, x_, h0_):
        h, last, _ = O.forward(a_, x_, off, h0_, reverse, coupled)
        return (h * dh).sum() + (last * dl).sum()

    _, _, before = O.forward(a, x, off, h0, reverse, coupled)
    got = O.backward(a, x, off, before, dh, dl, reverse, coupled)
    eps = 1e-4
    for n, v in enumerate((a, x, h0)):
        for i in np.ndindex(v.shape):
            args = [a.copy(), x.copy(), h0.copy()]
            args[n][i] += eps
            up = loss(*args)
            args[n][i] -= 2 * eps
            # the loss is multilinear along a sequence: differences of degree <= 7 terms
            assert abs((up - loss(*args)) / (2 * eps) - got[n][i]) <= 1e-6 * (1 + abs(got[n][i]))


def test_empty_sequences_pass_their_state():
    rng, off, a, x, h0 = _case(5)
    _, last, before = O.forward(a, x, off, h0)
    np.testing.assert_array_equal(last[1], h0[1])
    dl = rng.normal(size=h0.shape)
    np.testing.assert_array_equal(O.backward(a, x, off, before, None, dl)[2][1], dl[1])


def test_magnitude_recurrence_bounds_the_values():
    rng, off, a, x, h0 = _case(7)
    a = a * rng.choice([-1, 1], a.shape)
    h, last, b = O.forward(a, x, off, h0, coupled=True)
    hm, lastm, bm = O.forward(a, x, off, h0, coupled=True, magnitude=True)
    assert np.all(np.abs(h) <= hm + 1e-12) and np.all(np.abs(last) <= lastm + 1e-12)
    dh = rng.normal(size=x.shape)
    for g, gm in zip(O.backward(a, x, off, b, dh, None, False, True),
                     O.backward(a, x, off, bm, dh, None, False, True, magnitude=True)):
        assert np.all(np.abs(g) <= gm + 1e-12)
