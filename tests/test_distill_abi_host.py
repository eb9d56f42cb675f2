"""What distill refuses (no GPU needed): every argument error is reported on the host, before anything reaches
the device."""
import ctypes

import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L

from test_layer_abi_host import Fake


@pytest.fixture(scope="module", autouse=True)
def so():
    B.build()
    return L.load()


def _args(T=20):
    f, V, K = Fake(), 1000, 16
    a = dict(T=T, V=V, ld=1008, logits=f(T * 1008 * 2), dtype=M.LM_BF16, targets=f(T * 8), index=M.LM_I64, scale=1.0,
             t=dict(ids=f(T * K * 4), values=f(T * K * 4), K=K, index=M.LM_I32, dtype=M.LM_F32, rest=0))
    for n in ("kl", "logp", "lse", "dkl", "dlogp"):
        a[n] = f(T * 4)
    a["saved"], a["dlogits"], a["ld_out"] = f(T * 32), f(T * 1008 * 2), 1008
    return a


def _t(a):
    return None if a["t"] is None else ctypes.byref(M.lm_teacher(*[a["t"][n] for n, _ in M.lm_teacher._fields_]))


def _fwd(a):
    return M.call_status("distill_fwd", a["T"], a["V"], a["ld"], a["logits"], a["dtype"], _t(a), a["targets"], a["index"],
                         a["scale"], a["kl"], a["logp"], a["lse"], a["saved"], None)


def _bwd(a):
    return M.call_status("distill_bwd", a["T"], a["V"], a["ld"], a["logits"], a["dtype"], _t(a), a["targets"], a["index"],
                         a["scale"], a["saved"], a["dkl"], a["dlogp"], a["dlogits"], a["ld_out"], None)


@pytest.mark.parametrize("call,outs,ins", [(_fwd, ["kl", "logp", "lse", "saved"], ["logits", "targets"]),
                                           (_bwd, ["dlogits"], ["logits", "targets", "saved", "dkl", "dlogp"])])
def test_refusals(call, outs, ins):
    base = _args()

    def with_t(**kw):
        return dict(base, t=dict(base["t"], **kw))

    for n in ["logits", "t", "saved"] + (["kl", "logp", "lse"] if call is _fwd else ["dlogits"]):
        assert call(dict(base, **{n: None})) == L.LM_ERR_NULL, n
    for n in ("ids", "values"):
        assert call(with_t(**{n: None})) == L.LM_ERR_NULL, n
        assert call(with_t(**{n: base["t"][n] + 2})) == L.LM_ERR_ALIGN, n
    assert call(with_t(ids=base["t"]["ids"] + 4, index=M.LM_I64)) == L.LM_ERR_ALIGN
    for n in outs + ins:
        off = {"saved": 16, "targets": 4, "logits": 1, "dlogits": 1}.get(n, 2)
        assert call(dict(base, **{n: base[n] + off})) == L.LM_ERR_ALIGN, n
    for k, v in (("T", -1), ("T", 2 ** 31), ("V", 0), ("V", 2 ** 30 + 1), ("ld", 999), ("ld", 2 ** 41), ("scale", 0.0),
                 ("scale", -1.0), ("scale", float("inf")), ("scale", float("nan"))):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    for K in (0, -1, 129):
        assert call(with_t(K=K)) == L.LM_ERR_SHAPE, K
    for kw in (dict(index=2), dict(dtype=2)):
        assert call(with_t(**kw)) == L.LM_ERR_DTYPE, kw
        assert call(dict(base, **kw)) == L.LM_ERR_DTYPE, kw
    for out in outs:
        for other in outs + ins + ["ids", "values"]:
            if other != out and not (out == "dlogits" and other == "logits"):  # (in place is offered)
                at = base["t"][other] if other in base["t"] else base[other]
                assert call(dict(base, **{out: at})) in (L.LM_ERR_ALIAS, L.LM_ERR_ALIGN), (out, other)
    assert call(dict(base, targets=None)) == L.LM_ERR_SHAPE  # (logp, or dlogp, without targets)
    if call is _bwd:
        assert call(dict(base, ld_out=999)) == L.LM_ERR_SHAPE
        assert call(dict(base, dlogits=base["logits"], ld_out=1016)) == L.LM_ERR_ALIAS
        assert call(dict(base, dlogits=base["logits"] + 32)) == L.LM_ERR_ALIAS
    assert call(_args(T=0)) == L.LM_OK
    none = dict(_args(T=0), targets=None, logp=None, dlogp=None)
    assert call(none) == L.LM_OK


def test_the_binding_refuses():
    z, ids, v = torch.zeros(3, 10), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        M.distill_fwd(z, M.Teacher(ids, v))
    for t, err in ((M.Teacher(ids[0], v), TypeError), (M.Teacher(ids, v.double()), TypeError), (M.Teacher(ids.short(), v), TypeError)):
        with pytest.raises(err):
            t.c_struct(3)


def test_a_new_gradient_lies_like_its_logits():
    for dtype, w in ((torch.bfloat16, 8), (torch.float32, 4)):
        for T, V, ld, off in ((5, 33, 33, 0), (5, 33, 40, 3), (4, 7, 1000, 5), (1, 9, 9, 1), (0, 9, 9, 0)):
            x = torch.empty(8 + T * ld + ld, dtype=dtype)
            start = (-(x.data_ptr() // x.element_size())) % w + off
            z = x.as_strided((T, V), (ld, 1), start)
            d = M._alike(z)
            assert d.shape == (T, V) and d.stride(1) == 1 and (T < 2 or d.stride(0) >= V)
            if T > 1:
                assert (d.stride(0) - ld) % w == 0 and d.stride(0) <= 2 * V + 2 * w
            if T:
                assert (d.data_ptr() - z.data_ptr()) % 16 == 0
