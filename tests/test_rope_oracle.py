"""Pins of the rotary-position oracle (CPU): rotation as complex multiplication, row
norms, dependence of scores on position differences only, and gradients against
central differences."""
import numpy as np
import pytest

from oracle import rope_oracle as R

AXES, D = (8, 12, 10), 32


def _setup(pairs, seed=0, grid=(2, 3, 4), n_text=2):
    rng = np.random.default_rng(seed)
    pos = R.positions(grid, n_text, rng.normal(size=(n_text, 3)) * 7)
    return rng, R.angles(pos, AXES, D, 10000.0), rng.normal(size=(2, 3, pos.shape[0], D))


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_rotation_is_a_complex_product(pairs):
    _, ang, x = _setup(pairs)
    y = R.forward(x, ang, pairs)
    if pairs == "adjacent":
        zx, zy = x[..., 0::2] + 1j * x[..., 1::2], y[..., 0::2] + 1j * y[..., 1::2]
    else:
        zx, zy = x[..., :16] + 1j * x[..., 16:], y[..., :16] + 1j * y[..., 16:]
    np.testing.assert_allclose(zy, zx * np.exp(1j * ang), rtol=0, atol=1e-12)
    np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-12)
    # 15 of 16 pairs belong to an axis; the last one is left as it is
    np.testing.assert_array_equal(zy[..., 15], zx[..., 15])


def test_positions_and_angles():
    pos = R.positions((2, 2, 3), 1, None, origin=(5.0, 0.0, -1.0), step=(1.0, 0.5, 2.0))
    assert pos.shape == (13, 3)
    np.testing.assert_array_equal(pos[11], [6.0, 0.5, 3.0])
    ang = R.angles(pos, (2, 4, 2), 16, 100.0)
    np.testing.assert_allclose(ang[11], [6.0, 0.5, 0.5 * 100.0**-0.5, 3.0, 0, 0, 0, 0])
    assert not ang[12].any()  # a text row without a position is not turned


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_scores_depend_on_position_differences(pairs):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=D), rng.normal(size=D)
    a, b, move = rng.normal(size=(3, 1, 3)) * 20
    score = lambda p, r: (R.rotate(q[None], R.angles(p, AXES, D, 100.0), pairs)  # noqa: E731
                          * R.rotate(k[None], R.angles(r, AXES, D, 100.0), pairs)).sum()
    assert abs(score(a, b) - score(a + move, b + move)) < 1e-9
    assert abs(score(a, b) - score(a + move, b)) > 1e-3


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(pairs, norm):
    rng, ang, x = _setup(pairs)
    w = 1 + 0.3 * rng.normal(size=D) if norm else None
    dy = rng.normal(size=x.shape)
    loss = lambda x, w: (R.forward(x, ang, pairs, w, 1e-3) * dy).sum()  # noqa: E731
    dx, dw = R.backward(x, ang, pairs, dy, w, 1e-3)
    h = 1e-5
    for _ in range(20):
        i = tuple(rng.integers(n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in (0, 7, D - 1):
            e = np.zeros(D)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-6
