"""What cross attention refuses (no GPU needed): every argument error is reported on the host, before anything
reaches the device."""
import ctypes

import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L

from test_layer_abi_host import Fake, _ref, _size


@pytest.fixture(scope="module", autouse=True)
def so():
    B.build()
    return L.load()


def _args(Tq=300, Tk=200, hq=4, hk=2, d=64):
    f = Fake()
    a = dict(Tq=Tq, Tk=Tk, hq=hq, hk=hk, d=d)
    for n, T, h in (("q", Tq, hq), ("k", Tk, hk), ("v", Tk, hk), ("dO", Tq, hq)):
        a[n] = M.lm_heads(f(T * h * d * 2), h * d, d)
    a["a"] = dict(scale=0.125, cap=0.0, cu_q=f(64), cu_k=f(64), k_len=f(64), n_docs=3, reserved=0)
    for n, T, h in (("O", Tq, hq), ("dQ", Tq, hq), ("dK", Tk, hk), ("dV", Tk, hk)):
        a[n] = f(T * h * d * 2)
    a["O_lo"], a["lse"] = f(Tq * hq * d), f(Tq * hq * 4)
    a["ws_bytes"] = _size("cross_workspace_size", Tq, Tk, hq, hk, d)[1]
    a["ws"] = f(a["ws_bytes"])
    return a


def _a(a):
    return None if a["a"] is None else ctypes.byref(M.lm_cross(*[a["a"][n] for n, _ in M.lm_cross._fields_]))


def _fwd(a):
    return M.call_status("cross_fwd", a["Tq"], a["Tk"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _ref(a["v"]), _a(a),
                         a["O"], a["O_lo"], a["lse"], a["ws"], a["ws_bytes"], None)


def _bwd(a):
    return M.call_status("cross_bwd", a["Tq"], a["Tk"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _ref(a["v"]),
                         _ref(a["dO"]), a["O"], a["O_lo"], a["lse"], _a(a), a["dQ"], a["dK"], a["dV"], a["ws"], a["ws_bytes"], None)


def test_sizes():
    st, few = _size("cross_workspace_size", 1, 8192, 32, 8, 128)
    assert st == L.LM_OK and few >= 256 + 8193 * 8 + 38 * 32 * (128 + 2) * 4
    st, many = _size("cross_workspace_size", 2 ** 20, 2 ** 20, 8, 8, 128)  # (no parts: no megabytes for them)
    assert st == L.LM_OK and many < 2 ** 20 * (16 + 8 * 8) + 2 * 2 ** 20 // 8 + 2 ** 12  # (ranges, delta and lse; who is seen, by bits)
    for ok in ((0, 10, 4, 2, 64), (10, 0, 4, 2, 64), (0, 0, 4, 2, 64), (5, 5, 1024, 1, 8)):
        assert _size("cross_workspace_size", *ok)[0] == L.LM_OK, ok
    for bad in ((-1, 10, 4, 2, 64), (10, -1, 4, 2, 64), (2 ** 20 + 1, 10, 4, 2, 64), (10, 2 ** 20 + 1, 4, 2, 64), (10, 10, 4, 3, 64),
                (10, 10, 0, 1, 64), (10, 10, 1025, 1, 64), (10, 10, 4, 2, 12), (10, 10, 4, 2, 136)):
        assert _size("cross_workspace_size", *bad)[0] == L.LM_ERR_SHAPE, bad
    assert M.call_status("cross_workspace_size", 10, 10, 4, 2, 64, None) == L.LM_ERR_NULL


def test_parts_never_take_more_than_their_bound():
    """Items, splits and parts over many sizes: the partial rows stay below 2 x 152 tiles of 128 forward, and backward below
    152 tiles of keys, twice, and 4 x 152 tiles of queries."""
    for hq, hk in ((1, 1), (8, 2), (32, 8), (20, 4), (128, 1), (300, 1), (64, 64)):
        for Tq in (1, 2, 31, 33, 100, 500, 1500, 5000):
            for Tk in (1, 128, 129, 1000, 20000, 2 ** 20):
                st, n = _size("cross_workspace_size", Tq, Tk, hq, hk, 64)
                flat = 256 * 10 + (Tq + Tk) * 9 + (Tq + 128) * hq * 8
                assert st == L.LM_OK and n <= flat + 128 * 4 * max(2 * 152 * (64 + 2), (2 * 152 + 4 * 152) * 64), (hq, hk, Tq, Tk, n)


@pytest.mark.parametrize("call,outs,ins", [(_fwd, ["O", "O_lo", "lse", "ws"], ["q", "k", "v"]),
                                           (_bwd, ["dQ", "dK", "dV", "ws"], ["q", "k", "v", "dO", "O", "O_lo", "lse"])])
def test_refusals(call, outs, ins):
    base = _args()
    heads = [n for n in ins if isinstance(base[n], M.lm_heads)]
    plain = [n for n in outs + ins if n not in heads]

    def with_a(**kw):
        return dict(base, a=dict(base["a"], **kw))

    for n in heads + ["a"] + [n for n in plain if n != "O_lo"]:
        assert call(dict(base, **{n: None})) == L.LM_ERR_NULL, n
    for n in plain:
        assert call(dict(base, **{n: base[n] + 16})) == L.LM_ERR_ALIGN, n
    for n in heads:
        t = base[n]
        assert call(dict(base, **{n: M.lm_heads(t.p + 8, t.token_stride, t.head_stride)})) == L.LM_ERR_ALIGN, n
        for ts, hs in ((t.token_stride + 4, t.head_stride), (t.token_stride, t.head_stride + 4), (56, 64), (64, 56), (64, 0)):
            assert call(dict(base, **{n: M.lm_heads(t.p, ts, hs)})) == L.LM_ERR_SHAPE, (n, ts, hs)
    for k, v in (("Tq", -1), ("Tk", -1), ("Tk", 2 ** 20 + 1), ("hk", 3), ("d", 60), ("d", 136)):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    for kw in (dict(scale=0.0), dict(scale=-0.125), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0),
               dict(cap=2.0 ** -15), dict(cap=2.0 ** 13), dict(cap=float("nan")), dict(n_docs=0), dict(n_docs=-1), dict(n_docs=2 ** 30 + 1), dict(cu_q=None)):
        assert call(with_a(**kw)) == L.LM_ERR_SHAPE, kw
    assert call(with_a(cu_k=None)) == L.LM_ERR_NULL
    for n in ("cu_q", "cu_k", "k_len"):
        assert call(with_a(**{n: base["a"][n] + 2})) == L.LM_ERR_ALIGN, n
    assert call(dict(base, ws_bytes=base["ws_bytes"] - 1)) == L.LM_ERR_WORKSPACE
    for out in outs:
        for other in outs + ins:
            if other != out:
                at = base[other].p if other in heads else base[other]
                assert call(dict(base, **{out: at})) == L.LM_ERR_ALIAS, (out, other)
        for n in ("cu_q", "cu_k", "k_len"):
            assert call(dict(base, **{out: base["a"][n] // 32 * 32})) == L.LM_ERR_ALIAS, (out, n)
    none = dict(_args(Tq=0, Tk=0))
    assert call(none) == L.LM_OK


def test_the_binding_refuses():
    cu = torch.zeros(3, dtype=torch.int32)
    for a in (M.Cross(0.1, cu_q=cu), M.Cross(0.1, cu_k=cu), M.Cross(0.1, k_len=cu)):
        with pytest.raises(ValueError):
            a.c_struct()
