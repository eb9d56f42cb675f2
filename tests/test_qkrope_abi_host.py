"""What qkrope refuses (no GPU needed): every argument error is reported on the host, before anything reaches
the device."""
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


T, HQ, HK, DIM = 50, 4, 2, 64
FIELDS = [f[0] for f in M.lm_qkrope._fields_]


def _args():
    f = Fake()
    a = dict(T=T, hq=HQ, hk=HK, d=DIM)
    for n in ("q", "k", "dq", "dk", "q_out", "k_out", "dq_in", "dk_in"):
        h = HQ if "q" in n else HK
        a[n] = M.lm_heads(f(T * h * DIM * 2), h * DIM, DIM)
    a["r"] = dict(inv_freq=f(128), pos=f(T * 8 * 3), axis=f(128), w_q=f(256), w_k=f(256), factor=1.0, eps=1e-6, w_offset=0.0,
                  rot=64, axes=1, interleaved=0, norm=1, pos_index=L.LM_OK, w_dtype=M.LM_BF16, reserved=0)
    a["dw_q"], a["dw_k"] = f(256), f(256)
    a["ws_bytes"] = _size("qkrope_workspace_size", T, HQ, HK, DIM)[1]
    a["ws"] = f(a["ws_bytes"])
    return a


def _r(a):
    return None if a["r"] is None else ctypes.byref(M.lm_qkrope(*[a["r"][n] for n in FIELDS]))


def _fwd(a):
    return M.call_status("qkrope_fwd", a["T"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _r(a), _ref(a["q_out"]),
                         _ref(a["k_out"]), None)


def _bwd(a):
    return M.call_status("qkrope_bwd", a["T"], a["hq"], a["hk"], a["d"], _ref(a["q"]), _ref(a["k"]), _ref(a["dq"]), _ref(a["dk"]),
                         _r(a), _ref(a["dq_in"]), _ref(a["dk_in"]), a["dw_q"], a["dw_k"], a["ws"], a["ws_bytes"], None)


def test_sizes():
    assert _size("qkrope_workspace_size", T, HQ, HK, DIM)[0] == L.LM_OK
    assert _size("qkrope_workspace_size", 0, 1, 0, 256)[0] == L.LM_OK
    for bad in ((-1, 4, 2, 64), (2 ** 31, 4, 2, 64), (10, 0, 2, 64), (10, 4, -1, 64), (10, 1025, 2, 64), (10, 4, 1025, 64),
                (10, 4, 2, 0), (10, 4, 2, 12), (10, 4, 2, 264)):
        assert _size("qkrope_workspace_size", *bad)[0] == L.LM_ERR_SHAPE, bad
    assert M.call_status("qkrope_workspace_size", 10, 4, 2, 64, None) == L.LM_ERR_NULL


@pytest.mark.parametrize("call,heads", [(_fwd, ["q", "k", "q_out", "k_out"]), (_bwd, ["q", "k", "dq", "dk", "dq_in", "dk_in"])])
def test_refusals(call, heads):
    base = _args()

    def with_r(**kw):
        return dict(base, r=dict(base["r"], **kw))

    for n in heads + ["r"]:
        assert call(dict(base, **{n: None})) == L.LM_ERR_NULL, n
    for n in heads:
        t = base[n]
        assert call(dict(base, **{n: M.lm_heads(t.p + 8, t.token_stride, t.head_stride)})) == L.LM_ERR_ALIGN, n
        for ts, hs in ((t.token_stride + 4, t.head_stride), (t.token_stride, 60), (56, 64), (-64, 64), (64, 0)):
            assert call(dict(base, **{n: M.lm_heads(t.p, ts, hs)})) == L.LM_ERR_SHAPE, (n, ts, hs)
    for k, v in (("T", -1), ("hq", 0), ("hk", -1), ("d", 60), ("d", 264)):
        assert call(dict(base, **{k: v})) == L.LM_ERR_SHAPE, (k, v)
    for kw in (dict(rot=72), dict(rot=4), dict(rot=-8), dict(axes=0), dict(factor=float("nan")), dict(factor=float("inf")),
               dict(eps=0.0), dict(eps=float("inf")), dict(w_offset=float("nan")), dict(rot=0),  # (pos and the others given)
               dict(norm=0)):                                                                    # (weights given)
        assert call(with_r(**kw)) == L.LM_ERR_SHAPE, kw
    nothing = dict(rot=0, norm=0, inv_freq=None, pos=None, axis=None, w_q=None, w_k=None)
    assert call(with_r(**nothing)) == L.LM_ERR_SHAPE
    for kw in (dict(pos_index=2), dict(w_dtype=2)):
        assert call(with_r(**kw)) == L.LM_ERR_DTYPE, kw
    for kw in (dict(inv_freq=None), dict(axes=3, axis=None), dict(axes=3, pos=None)):
        assert call(with_r(**kw)) == L.LM_ERR_NULL, kw
    r = base["r"]
    for kw in (dict(inv_freq=r["inv_freq"] + 2), dict(pos=r["pos"] + 2), dict(pos=r["pos"] + 4, pos_index=1), dict(axis=r["axis"] + 2),
               dict(w_q=r["w_q"] + 1), dict(w_k=r["w_k"] + 2, w_dtype=1)):
        assert call(with_r(**kw)) == L.LM_ERR_ALIGN, kw
    # no keys: nothing of theirs
    gone = {n: None for n in heads if "k" in n}
    assert call(dict(base, hk=0)) == L.LM_ERR_SHAPE
    if call is _fwd:
        assert call(dict(base, hk=0, **gone)) == L.LM_ERR_SHAPE  # (w_k)


def _moved(t, to, **kw):
    return M.lm_heads(to, kw.get("ts", t.token_stride), kw.get("hs", t.head_stride))


def test_what_may_overlap():
    """Calls that pass the checks end at the device's (there is none, or it is not asked): anything but LM_ERR_ALIAS."""
    base = _args()
    q, k = base["q"], base["k"]
    alias = lambda call, **kw: call(dict(base, **kw)) == L.LM_ERR_ALIAS  # noqa: E731
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    assert not alias(_fwd, q_out=q, k_out=k) and not alias(_bwd, dq_in=base["dq"], dk_in=base["dk"])
    assert alias(_fwd, q_out=_moved(q, q.p + 16)) and alias(_fwd, q_out=_moved(q, q.p, ts=q.token_stride + 64))
    assert alias(_fwd, q_out=k) and alias(_fwd, k_out=q) and alias(_bwd, dq_in=q) and alias(_bwd, dk_in=k)
    assert alias(_bwd, dq_in=base["dk"])
    # slices of one buffer of 8 heads: q 4, k 2, others 2
    row = 8 * DIM
    at = lambda head: M.lm_heads(q.p, row, DIM) if head == 0 else M.lm_heads(q.p + head * DIM * 2, row, DIM)  # noqa: E731
    assert not alias(_fwd, q=at(0), k=at(4), q_out=at(0), k_out=at(4))
    assert alias(_fwd, q=at(0), k=at(4), q_out=at(4), k_out=at(0)) and alias(_fwd, q=at(0), k=at(3), q_out=at(0))
    assert not alias(_fwd, q=at(0), k=at(4), k_out=at(6)) and alias(_fwd, q=at(0), k=at(4), k_out=at(7))
    # head-major: T x d per head
    col = lambda head: M.lm_heads(q.p + head * T * DIM * 2, DIM, T * DIM)  # noqa: E731
    assert not alias(_fwd, q=col(0), k=col(4), q_out=col(0), k_out=col(4)) and alias(_fwd, q=col(0), k=col(3), q_out=col(0), k_out=col(5))
    # an output whose own rows overlap
    assert alias(_fwd, q_out=M.lm_heads(base["q_out"].p, DIM, DIM))
    # flat buffers
    for n in ("dw_q", "dw_k", "ws"):
        assert alias(_bwd, dq_in=_moved(q, base[n])) and alias(_bwd, **{n: q.p}), n
    assert alias(_bwd, dw_q=base["dw_k"]) and alias(_bwd, dw_q=base["ws"])
    for n in ("inv_freq", "pos", "w_q"):
        assert alias(_fwd, k_out=_moved(k, base["r"][n])), n


def test_backward_refuses():
    base = _args()
    for n in ("dw_q", "dw_k"):
        assert _bwd(dict(base, **{n: base[n] + 2})) == L.LM_ERR_ALIGN
    assert _bwd(dict(base, ws=None)) == L.LM_ERR_NULL and _bwd(dict(base, ws=base["ws"] + 16)) == L.LM_ERR_ALIGN
    assert _bwd(dict(base, ws_bytes=base["ws_bytes"] - 1)) == L.LM_ERR_WORKSPACE
    off = dict(base["r"], norm=0, w_q=None, w_k=None)
    for n in ("dw_q", "dw_k"):
        only = dict(base, r=off, dw_q=None, dw_k=None)
        assert _bwd(dict(only, **{n: base[n]})) == L.LM_ERR_SHAPE


def test_the_binding_refuses():
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    r = M.QkRope(norm=True)
    for call in (lambda: M.qkrope_fwd(q, k, r), lambda: M.qkrope_bwd(q, k, q, k, r)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    with pytest.raises(ValueError):
        M.QkRope(pos=torch.zeros(5, dtype=torch.int32)).c_struct(5, 64)
