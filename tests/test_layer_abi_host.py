"""What the layer operators refuse (no GPU needed): every argument error is reported on the host before
anything reaches the device, in the C ABI and in the Python binding, and the library exports the header."""
import ctypes

import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L


@pytest.fixture(scope="module", autouse=True)
def so():
    B.build()
    return L.load()


def _size(fn, *args):
    out = ctypes.c_size_t(0)
    return M.call_status(fn, *args, ctypes.byref(out)), out.value


class Fake:
    """Distinct aligned addresses in place of device buffers; none is ever dereferenced."""

    def __init__(self):
        self.next = 1 << 32

    def __call__(self, nbytes):
        p = self.next
        self.next += (int(nbytes) + 4095) // 4096 * 4096 + 4096
        return p


def test_exports_every_header_symbol(so):
    names = M.header_symbols()
    for n in names:
        assert hasattr(so, n), n
    assert len(names) == len(set(names)) and set(names) == set(M._SIGS)
    assert not set(names) & set(L._SIGS)


def test_size_queries():
    st, s1 = _size("attn_workspace_size", 300, 4, 2, 64)
    assert st == L.LM_OK and s1 >= 256 + 300 * 16 + 2 * 384 * 4 * 4
    assert _size("attn_workspace_size", 301, 4, 2, 64)[1] >= s1
    assert _size("attn_workspace_size", 0, 4, 2, 64)[0] == L.LM_OK
    for bad in ((-1, 4, 2, 64), (2 ** 20 + 1, 4, 2, 64), (10, 4, 3, 64), (10, 0, 1, 64), (10, 4, 0, 64), (10, 1025, 1, 64),
                (10, 4, 2, 0), (10, 4, 2, 12), (10, 4, 2, 136)):
        assert _size("attn_workspace_size", *bad)[0] == L.LM_ERR_SHAPE, bad
    assert M.call_status("attn_workspace_size", 10, 4, 2, 64, None) == L.LM_ERR_NULL
    st, s1 = _size("addnorm_workspace_size", 300, 256)
    assert st == L.LM_OK and s1 >= 256 + 3 * 256 * 4
    for bad in ((-1, 256), (10, 16), (10, 40), (10, 16416), (2 ** 31, 256)):
        assert _size("addnorm_workspace_size", *bad)[0] == L.LM_ERR_SHAPE, bad
    assert M.call_status("addnorm_workspace_size", 10, 256, None) == L.LM_ERR_NULL
    for mask in (-1, 8):
        assert M.call_status("attn_debug_inject", mask, 0) == L.LM_ERR_SHAPE


# ------------------------------------------------------------------------------------ attention
def _attn_args(T=300, hq=4, hk=2, d=64):
    f = Fake()
    a = dict(T=T, hq=hq, hk=hk, d=d)
    for n, h in (("q", hq), ("k", hk), ("v", hk), ("dO", hq)):
        a[n] = M.lm_heads(f(T * h * d * 2), h * d, d)
    a["a"] = M.lm_attn(0.125, 0.0, 0, 1, 0, f(64), 0, 3, 0)
    for n, h in (("O", hq), ("dQ", hq), ("dK", hk), ("dV", hk)):
        a[n] = f(T * h * d * 2)
    a["O_lo"], a["lse"] = f(T * hq * d), f(T * hq * 4)
    a["ws_bytes"] = _size("attn_workspace_size", T, hq, hk, d)[1]
    a["ws"] = f(a["ws_bytes"])
    return a


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _attn_fwd(a):
    return M.call_status("attn_fwd", a["T"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _ref(a["v"]), _ref(a["a"]),
                         a["O"], a["O_lo"], a["lse"], a["ws"], a["ws_bytes"], None)


def _attn_bwd(a):
    return M.call_status("attn_bwd", a["T"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _ref(a["v"]),
                         _ref(a["dO"]), a["O"], a["O_lo"], a["lse"], _ref(a["a"]), a["dQ"], a["dK"], a["dV"], a["ws"],
                         a["ws_bytes"], None)


@pytest.mark.parametrize("call,outs,ins", [(_attn_fwd, ["O", "O_lo", "lse", "ws"], ["q", "k", "v"]),
                                           (_attn_bwd, ["dQ", "dK", "dV", "ws"], ["q", "k", "v", "dO", "O", "O_lo", "lse"])])
def test_attention_refuses(call, outs, ins):
    base = _attn_args()
    heads = [n for n in ins if isinstance(base[n], M.lm_heads)]
    plain = [n for n in outs + ins if n not in heads]
    for n in heads + ["a"] + [n for n in plain if n != "O_lo"]:
        assert call(dict(base, **{n: None})) == L.LM_ERR_NULL, n
    for n in plain:
        assert call(dict(base, **{n: base[n] + 16})) == L.LM_ERR_ALIGN, n
    for n in heads:
        t = base[n]
        assert call(dict(base, **{n: M.lm_heads(t.p + 8, t.token_stride, t.head_stride)})) == L.LM_ERR_ALIGN, n
        assert call(dict(base, **{n: M.lm_heads(None, t.token_stride, t.head_stride)})) == L.LM_ERR_NULL, n
        for ts, hs in ((t.token_stride + 4, t.head_stride), (t.token_stride, t.head_stride + 4), (56, 64), (64, 56),
                       (-64, 64), (64, 0), (2 ** 39, 64)):
            assert call(dict(base, **{n: M.lm_heads(t.p, ts, hs)})) == L.LM_ERR_SHAPE, (n, ts, hs)
    for k, v in (("T", -1), ("T", 2 ** 20 + 1), ("hk", 3), ("hk", 0), ("hq", 0), ("d", 60), ("d", 136), ("d", 0)):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    assert call(dict(base, ws_bytes=base["ws_bytes"] - 1)) == L.LM_ERR_WORKSPACE
    for n in outs:  # results may not lie on inputs or on one another
        for other in heads:
            assert call(dict(base, **{n: base[other].p + 64})) == L.LM_ERR_ALIAS, (n, other)
        for other in plain:
            if other != n:
                assert call(dict(base, **{n: base[other]})) == L.LM_ERR_ALIAS, (n, other)
    docs = base["a"].cu_docs
    inf, nan = float("inf"), float("nan")
    for a, st in ((M.lm_attn(nan, 0, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE), (M.lm_attn(inf, 0, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE),
                  (M.lm_attn(1, -1, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE), (M.lm_attn(1, inf, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE),
                  (M.lm_attn(1, 2.0 ** 13, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE), (M.lm_attn(1, 1e-30, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE),
                  (M.lm_attn(1e38, 1e-3, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE),
                  (M.lm_attn(1, nan, 0, 1, 0, docs, 0, 3, 0), L.LM_ERR_SHAPE), (M.lm_attn(1, 0, 0, 1, -1, docs, 0, 3, 0), L.LM_ERR_SHAPE),
                  (M.lm_attn(1, 0, 0, 1, 0, docs, 0, 0, 0), L.LM_ERR_SHAPE),       # offsets of no document
                  (M.lm_attn(1, 0, 0, 1, 0, 0, docs, 3, 0), L.LM_ERR_SHAPE),       # a prefix without documents
                  (M.lm_attn(1, 0, docs + 2, 1, 0, 0, 0, 0, 0), L.LM_ERR_ALIGN), (M.lm_attn(1, 0, 0, 1, 0, docs + 2, 0, 3, 0), L.LM_ERR_ALIGN),
                  (M.lm_attn(1, 0, 0, 1, 0, docs, docs + 2, 3, 0), L.LM_ERR_ALIGN)):
        assert call(dict(base, a=a)) == st
    assert call(dict(_attn_args(T=0))) == L.LM_OK  # no tokens: nothing to do


# ------------------------------------------------------------------------------------ addnorm
def _addnorm_args(T=300, d=256):
    f = Fake()
    a = dict(T=T, d=d)
    for n in ("h", "y", "dh_out", "dx", "h_out", "x", "dh", "dy"):
        a[n] = f(T * d * 4)
    for n in ("rstd_y", "rstd_h"):
        a[n] = f(T * 4)
    for n in ("dw_in", "dw_post", "dgate"):
        a[n] = f(d * 4)
    a["n"] = M.lm_addnorm(f(d * 4), f(d * 4), f(d * 4), 1.0, 1e-5, 0.0, M.LM_F32, M.LM_F32, 0)
    a["ws_bytes"] = _size("addnorm_workspace_size", T, d)[1]
    a["ws"] = f(a["ws_bytes"])
    return a


def _addnorm_fwd(a):
    return M.call_status("addnorm_fwd", a["T"], a["d"], a["h"], a["y"], _ref(a["n"]), a["h_out"], a["x"], a["rstd_y"],
                         a["rstd_h"], None)


def _addnorm_bwd(a):
    return M.call_status("addnorm_bwd", a["T"], a["d"], a["h"], a["y"], a["dh_out"], a["dx"], a["rstd_y"], a["rstd_h"],
                         _ref(a["n"]), a["dh"], a["dy"], a["dw_in"], a["dw_post"], a["dgate"], a["ws"], a["ws_bytes"], None)


def _norm(n, **over):
    fields = {f: getattr(n, f) for f, _ in M.lm_addnorm._fields_}
    return M.lm_addnorm(**dict(fields, **over))


@pytest.mark.parametrize("call,outs,ins,may_be_null",
                         [(_addnorm_fwd, ["h_out", "x", "rstd_y", "rstd_h"], ["h", "y"], []),
                          (_addnorm_bwd, ["dh", "dy", "dw_in", "dw_post", "dgate", "ws"],
                           ["h", "y", "dh_out", "dx", "rstd_y", "rstd_h"], ["dh_out", "dw_in", "dw_post", "dgate"])])
def test_addnorm_refuses(call, outs, ins, may_be_null):
    base = _addnorm_args()
    n = base["n"]
    for name in outs + ins + ["n"]:
        if name not in may_be_null + ["y"]:
            assert call(dict(base, **{name: None})) == L.LM_ERR_NULL, name
    for name in outs + ins:
        assert call(dict(base, **{name: base[name] + 16})) == L.LM_ERR_ALIGN, name
    for k, v in (("T", -1), ("T", 2 ** 31), ("d", 16), ("d", 260), ("d", 16416)):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    for out in outs:
        for other in outs + ins:
            if other != out:
                assert call(dict(base, **{out: base[other]})) == L.LM_ERR_ALIAS, (out, other)
        for w in ("w_in", "w_post", "gate"):
            assert call(dict(base, **{out: getattr(n, w)})) == L.LM_ERR_ALIAS, (out, w)
    for over, st in (({"h_dtype": 2}, L.LM_ERR_DTYPE), ({"w_dtype": -1}, L.LM_ERR_DTYPE), ({"eps": 0.0}, L.LM_ERR_SHAPE),
                     ({"eps": float("inf")}, L.LM_ERR_SHAPE), ({"eps": float("nan")}, L.LM_ERR_SHAPE),
                     ({"alpha": float("nan")}, L.LM_ERR_SHAPE), ({"w_offset": float("inf")}, L.LM_ERR_SHAPE),
                     ({"w_in": n.w_in + 16}, L.LM_ERR_ALIGN), ({"w_post": n.w_post + 16}, L.LM_ERR_ALIGN),
                     ({"gate": n.gate + 16}, L.LM_ERR_ALIGN)):
        assert call(dict(base, n=_norm(n, **over))) == st, over
    assert call(dict(base, y=None)) == L.LM_ERR_SHAPE                                         # a norm of nothing
    assert call(dict(base, y=None, n=_norm(n, w_post=None))) == L.LM_ERR_SHAPE                # a gate of nothing
    assert call(dict(base, y=None, n=_norm(n, w_in=None, w_post=None, gate=None))) == L.LM_ERR_NULL  # nothing to do
    if call is _addnorm_bwd:
        assert call(dict(base, ws_bytes=base["ws_bytes"] - 1)) == L.LM_ERR_WORKSPACE
        for w, grad in (("w_in", "dw_in"), ("w_post", "dw_post"), ("gate", "dgate")):         # of a missing vector
            a = dict(base, n=_norm(n, **{w: None}), dx=None if w == "w_in" else base["dx"])
            assert call(a) == L.LM_ERR_SHAPE and grad in L.last_error()
        assert call(dict(base, n=_norm(n, w_in=None), dw_in=None)) == L.LM_ERR_SHAPE          # dx without w_in
    else:
        assert call(_addnorm_args(T=0)) == L.LM_OK


# ------------------------------------------------------------------------------------ logprob
def _logprob_args(T=300, V=1000, k=5):
    f = Fake()
    a = dict(T=T, V=V, ld=V, dtype=M.LM_BF16, index=M.LM_I64, scale=1.0, k=k, ld_out=V)
    a["logits"], a["dlogits"], a["targets"] = f(T * V * 2), f(T * V * 2), f(T * 8)
    for n in ("logp", "entropy", "lse", "dlogp", "dentropy"):
        a[n] = f(T * 4)
    a["top_ids"], a["top_logp"] = f(T * k * 4), f(T * k * 4)
    return a


def _logprob_fwd(a):
    return M.call_status("logprob_fwd", a["T"], a["V"], a["ld"], a["logits"], a["dtype"], a["targets"], a["index"], a["scale"],
                         a["k"], a["logp"], a["entropy"], a["lse"], a["top_ids"], a["top_logp"], None)


def _logprob_bwd(a):
    return M.call_status("logprob_bwd", a["T"], a["V"], a["ld"], a["logits"], a["dtype"], a["targets"], a["index"], a["scale"],
                         a["lse"], a["entropy"], a["dlogp"], a["dentropy"], a["dlogits"], a["ld_out"], None)


@pytest.mark.parametrize("call,outs,ins,may_be_null",
                         [(_logprob_fwd, ["logp", "entropy", "lse", "top_ids", "top_logp"], ["logits", "targets"], ["entropy"]),
                          (_logprob_bwd, ["dlogits"], ["logits", "targets", "lse", "entropy", "dlogp", "dentropy"],
                           ["dlogp", "dentropy"])])
def test_logprob_refuses(call, outs, ins, may_be_null):
    base = _logprob_args()
    for n in outs + ins:
        if n not in may_be_null:
            assert call(dict(base, **{n: None})) == L.LM_ERR_NULL, n
        assert call(dict(base, **{n: base[n] + 1})) == L.LM_ERR_ALIGN, n
    assert call(dict(base, targets=base["targets"] + 4)) == L.LM_ERR_ALIGN
    assert call(dict(base, dtype=M.LM_F32, logits=base["logits"] + 2)) == L.LM_ERR_ALIGN
    for k, v in (("T", -1), ("T", 2 ** 31), ("V", 0), ("V", 2 ** 30 + 1), ("ld", 999), ("scale", 0.0), ("scale", -1.0),
                 ("scale", float("inf")), ("scale", float("nan"))):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    for k in ("dtype", "index"):
        assert call(dict(base, **{k: 2})) == L.LM_ERR_DTYPE, k
    for out in outs:
        for other in outs + ins:
            if other != out and not (out == "dlogits" and other == "logits"):  # (in place is offered)
                assert call(dict(base, **{out: base[other]})) == L.LM_ERR_ALIAS, (out, other)
    if call is _logprob_fwd:
        for over in ({"k": 33}, {"k": -1}, {"k": 5, "V": 4, "ld": 4}, {"k": 0}, {"k": 0, "top_ids": None}):
            assert call(dict(base, **over)) == L.LM_ERR_SHAPE, over
    else:
        assert call(dict(base, ld_out=999)) == L.LM_ERR_SHAPE
        assert call(dict(base, dlogits=base["logits"], ld_out=1008)) == L.LM_ERR_ALIAS    # rows would move
        assert call(dict(base, dlogits=base["logits"] + 32)) == L.LM_ERR_ALIAS
        assert call(dict(_logprob_args(T=0), dlogits=base["dlogits"])) == L.LM_OK
    assert call(_logprob_args(T=0)) == L.LM_OK


# ------------------------------------------------------------------------------------ the binding
def test_the_binding_refuses_what_is_not_on_the_device_or_of_another_type():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        M._heads(x, 4, 2, 64, "q")
    with pytest.raises(TypeError, match="torch.Tensor"):
        M._heads(np.zeros((4, 2, 64)), 4, 2, 64, "q")
    with pytest.raises(ValueError, match="CUDA"):
        M._shaped(torch.zeros(3), (3,), torch.float32, "lse")
    with pytest.raises(TypeError, match="torch.Tensor"):
        M._shaped([0.0], (1,), torch.float32, "lse")
    with pytest.raises(TypeError, match="2D"):
        M._rows2d(torch.zeros(3), "logits")
    with pytest.raises(ValueError, match="CUDA"):
        M._rows2d(torch.zeros(3, 4), "logits")
    with pytest.raises(TypeError, match="int32 or int64"):
        M._targets(torch.zeros(3), 3)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        M.AddNorm().c_struct(64, torch.float16)
    with pytest.raises(L.LmError, match="d = 12"):
        M.attn_workspace_size(10, 4, 2, 12)
