"""The fp64 definitions of the layer operators (oracle/layer.py): gradients against central differences
of the forward, masks against their description, and values that can be worked out by hand."""
import numpy as np
import pytest

from oracle import layer as O


def _rng(seed):
    return np.random.default_rng(seed)


def _central(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + eps
        a = f()
        x[i] = old - eps
        b = f()
        x[i] = old
        g[i] = (a - b) / (2 * eps)
    return g


# central differences in fp64 with eps = 1e-5: truncation O(eps^2) times third derivatives of order one,
# rounding about 1e-16 / 1e-5 times values of order ten
DIFF_TOL = 1e-8


@pytest.mark.parametrize("cap,bias,kw", [
    (0.0, False, {}), (2.0, False, {}), (0.0, True, {"causal": False}), (1.5, True, {"window": 3}),
    (2.0, False, {"cu_docs": [0, 0, 3, 4, 7], "prefix": [0, 2, 1, 3]}), (0.0, True, {"cu_docs": [1, 5, 6]})])
def test_attention_gradients_match_differences(cap, bias, kw):
    g = _rng(3)
    T, hq, hk, d = 8, 4, 2, 3
    q, k, v, dO = (g.standard_normal((T, h, d)) for h in (hq, hk, hk, hq))
    see = O.visible(T, **kw)
    slopes = np.array([0.5, 0.25, 0.1, 0.0]) if bias else None

    def f():
        return float((O.attn_forward(q, k, v, see, 0.7, cap, slopes)["O"] * dO).sum())

    got = O.attn_backward(q, k, v, dO, see, 0.7, cap, slopes)
    for name, x in (("dQ", q), ("dK", k), ("dV", v)):
        assert np.abs(got[name] - _central(f, x)).max() < DIFF_TOL, name


def test_visible_intervals():
    see = O.visible(10, causal=True, window=0, cu_docs=[1, 4, 4, 9], prefix=[2, 0, 3])
    rows = {0: [], 1: [1, 2], 2: [1, 2], 3: [1, 2, 3], 4: [4, 5, 6], 5: [4, 5, 6], 6: [4, 5, 6], 7: [4, 5, 6, 7],
            8: [4, 5, 6, 7, 8], 9: []}
    for i, js in rows.items():
        assert list(np.flatnonzero(see[i])) == js, i
    assert list(np.flatnonzero(O.visible(6, causal=False, window=2)[3])) == [2, 3, 4]


def test_attention_row_that_sees_one_key_or_none():
    g = _rng(5)
    q, k, v = (g.standard_normal((3, 1, 4)) for _ in range(3))
    out = O.attn_forward(q, k, v, O.visible(3, cu_docs=[0, 1, 2]), 1.0, 0.0, np.array([2.0]))
    assert np.array_equal(out["O"][:2], v[:2])
    assert np.all(out["O"][2] == 0) and np.isneginf(out["lse"][0, 2])
    assert np.allclose(out["lse"][0, :2], (q[:2, 0] * k[:2, 0]).sum(1))


@pytest.mark.parametrize("add,post,gate,inn", [(1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 0), (0, 0, 0, 1), (1, 0, 0, 1)])
def test_addnorm_gradients_match_differences(add, post, gate, inn):
    g = _rng(7)
    T, d = 3, 5
    h = g.standard_normal((T, d))
    y = g.standard_normal((T, d)) if add else None
    w_in, w_post, gt = (g.standard_normal(d) if on else None for on in (inn, post, gate))
    dh, dx = g.standard_normal((T, d)), g.standard_normal((T, d)) if inn else None

    def f():
        o = O.addnorm_forward(h, y, w_in, w_post, gt, 0.7, 1e-3, 0.5)
        return float((o["h"] * dh).sum() + ((o["x"] * dx).sum() if inn else 0.0))

    got = O.addnorm_backward(h, y, dh, dx, w_in, w_post, gt, 0.7, 1e-3, 0.5)
    for name, x in (("dh", h), ("dy", y), ("dw_in", w_in), ("dw_post", w_post), ("dgate", gt)):
        if x is None:
            assert got[name] is None
        else:
            assert np.abs(got[name] - _central(f, x)).max() < DIFF_TOL, name


def test_logprob_gradients_match_differences():
    g = _rng(9)
    T, V = 4, 7
    x = g.standard_normal((T, V)) * 2
    x[1, 3] = -np.inf
    t = np.array([2, -100, 6, 0])
    gl, ge = g.standard_normal(T), g.standard_normal(T)

    def f():
        o = O.logprob_forward(x, t, 0, 1.3)
        return float((o["logp"] * gl).sum() + (o["entropy"] * ge).sum())

    got = O.logprob_backward(x, t, gl, ge, 1.3)
    assert got[1, 3] == 0
    x[1, 3] = -800.0  # (differences of an infinite entry do not exist; its probability is zero all the same)
    assert np.abs(got - _central(f, x)).max() < DIFF_TOL


def test_logprob_ties_and_empty_rows():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 3.0], [-np.inf] * 5, [0.0, -0.0, np.nan, 0.0, 1.0]])
    o = O.logprob_forward(x, np.array([1, 0, 9]), 4)
    assert o["top_ids"][0].tolist() == [1, 2, 4, 0] and o["top_ids"][2].tolist() == [2, 4, 0, 1]
    assert np.isneginf(o["lse"][1]) and np.isneginf(o["logp"][1]) and o["entropy"][1] == 0 and o["logp"][2] == 0
    assert np.all(O.logprob_backward(x[:2], np.array([1, 0]), np.ones(2), np.ones(2))[1] == 0)
    u = O.logprob_forward(np.zeros((1, 8)), np.array([3]))
    assert np.isclose(u["entropy"][0], np.log(8)) and np.isclose(u["logp"][0], -np.log(8))
