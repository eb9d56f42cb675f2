"""The fp64 definition of distillation from a teacher's top logits: gradients against differences, and what
follows from the formulas."""
import numpy as np
import pytest

from oracle import layer as O


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("scale", [1.0, 0.6])
@pytest.mark.parametrize("hard", [False, True])
def test_gradients_against_differences(rest, scale, hard):
    g = np.random.default_rng(4)
    T, V, K = 6, 9, 4
    z = g.normal(size=(T, V)) * 2
    ids = np.array([[0, 3, 8, 5], [1, 1, 2, 4], [-1, 7, 9, 6], [-1, -1, -1, -1], [2, 0, 1, 3], [5, 5, 5, 5]])
    values = np.log(g.dirichlet(np.ones(K + 1), size=T))[:, :K] if rest else g.normal(size=(T, K))
    values[4, 1] = -np.inf
    targets = np.array([3, -100, 0, 8, 9, 5]) if hard else None
    dkl, dlogp = g.normal(size=T), g.normal(size=T) if hard else None

    def f(z):
        o = O.distill_forward(z, ids, values, targets, scale, rest)
        return (dkl * o["kl"]).sum() + (0.0 if not hard else (dlogp * o["logp"]).sum())

    d = O.distill_backward(z, ids, values, dkl, targets, dlogp, scale, rest)
    for i in np.ndindex(z.shape):
        e = np.zeros_like(z)
        e[i] = 1e-6
        assert abs((f(z + e) - f(z - e)) / 2e-6 - d[i]) < 1e-7, i


def test_a_whole_teacher_is_the_divergence_and_its_own_student_has_none():
    g = np.random.default_rng(5)
    z, y = g.normal(size=(3, 8)), g.normal(size=(3, 8))
    ids = np.tile(np.arange(8), (3, 1))
    got = O.distill_forward(z, ids, y)["kl"]
    lp, lq = (x - np.log(np.exp(x).sum(1, keepdims=True)) for x in (y, z))
    assert np.allclose(got, (np.exp(lp) * (lp - lq)).sum(1), atol=1e-12)
    assert np.allclose(O.distill_forward(z, ids, z)["kl"], 0, atol=1e-12)
    # with the rest, the student's own top entries have no divergence and no gradient
    same = O.distill_forward(z, ids[:, :3], lq[:, :3], rest=True)["kl"]
    assert np.allclose(same, 0, atol=1e-12)
    assert np.allclose(O.distill_backward(z, ids[:, :3], lq[:, :3], np.ones(3), rest=True), 0, atol=1e-12)


def test_rows_without_entries_or_without_logits():
    z = np.full((3, 5), -np.inf)
    z[0] = [0.0, 1.0, -np.inf, 2.0, 0.0]
    ids, v = np.array([[-1, 7], [1, 2], [-1, -1]]), np.zeros((3, 2))
    o = O.distill_forward(z, ids, v, np.array([2, 1, 0]))
    assert o["kl"][0] == 0 and np.isposinf(o["kl"][1]) and o["kl"][2] == 0 and np.isneginf(o["logp"]).all()
    assert not O.distill_backward(z, ids, v, np.ones(3))[1:].any()
