"""The fp64 definition of the head norms with rotation: gradients against differences, a rotation's
properties, far positions."""
import numpy as np
import pytest

from oracle import layer as O


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_gradients_against_differences(norm, inter, rot):
    if not norm and not rot:
        return
    g = np.random.default_rng(1)
    T, h, d = 3, 2, 8
    x, dy, w = g.normal(size=(T, h, d)), g.normal(size=(T, h, d)), 1 + 0.1 * g.normal(size=d)
    a = O.qkrope_angles(T, 0.7 ** np.arange(rot // 2), np.array([0, 5, 11])) if rot else None
    kw = dict(angles=a, interleaved=inter, factor=1.3, norm=norm, eps=1e-2, w_offset=0.5)
    f = lambda x, w: (O.qkrope_forward(x, w=w if norm else None, **kw) * dy).sum()  # noqa: E731
    dx, dw = O.qkrope_backward(x, dy, w=w if norm else None, **kw)
    step = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - dx[i]) < 1e-7
    if norm:
        for i in range(d):
            e = np.zeros(d)
            e[i] = step
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * step) - dw[i]) < 1e-7


def test_scores_depend_on_the_distance_alone():
    g = np.random.default_rng(2)
    q, k = g.normal(size=(1, 1, 16)), g.normal(size=(1, 1, 16))
    f = 1e4 ** (-np.arange(8) / 8)

    def score(i, j):
        a, b = (O.qkrope_forward(x, O.qkrope_angles(1, f, [p])) for x, p in ((q, i), (k, j)))
        return (a * b).sum()

    assert abs(score(7, 3) - score(1007, 1003)) < 1e-10
    assert abs(score(0, 0) - (q * k).sum()) < 1e-12


def test_axes_turn_their_own_pairs():
    g = np.random.default_rng(3)
    x = g.normal(size=(5, 2, 12))
    f, pos = np.array([1.0, 0.5, 0.25, 1.0, 0.5, 0.25]), g.integers(0, 100, size=(3, 5))
    axis = np.array([0, 0, 1, 1, 2, 2])
    got = O.qkrope_forward(x, O.qkrope_angles(5, f, pos, axis))
    for p in range(6):
        one = O.qkrope_forward(x, O.qkrope_angles(5, f, pos[axis[p]]))
        assert np.array_equal(got[..., [p, p + 6]], one[..., [p, p + 6]])
