"""Attention to the states of another length (cross_fwd, cross_bwd) against the fp64 definition: lengths around the
128-token tiles on both sides, single queries and batches of them, segments that are empty, padded or hold NaN
where nothing looks, head layouts, strides, capped scores, gradients, captured and on other streams.

Tolerances as for attention over packed documents: rounded to bf16 are, for O: P and the result; for dV the same; for
dQ and dK: P (inside delta), the score gradient and the result.  A rounding moves a value by at most 2^-8 of
itself, 2^-8 / sqrt(3) in the mean square; three independent ones give 2^-8, and 1.5 times that, 3 x 2^-9, bounds the
relative Frobenius error.  lse is fp32 throughout: a score's error is at most a few 2^-24 of sum |q_i k_i|, below 2e-5
at these sizes; the parts of the keys add a rounding each of their sum's logarithm."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import check, host64

pytestmark = pytest.mark.gpu

REL = 3 * 2.0 ** -9
LSE_ABS = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _bf(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16().cuda()


def _int32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _make(Tq, Tk, hq, hk, d, cap=0.0, cu_q=None, cu_k=None, k_len=None, seed=0, std=2.0):
    x = _bf((Tq, hq, d), seed, std), _bf((Tk, hk, d), seed + 1), _bf((Tk, hk, d), seed + 2), _bf((Tq, hq, d), seed + 3)
    a = M.Cross(d ** -0.5, cap, _int32(cu_q), _int32(cu_k), _int32(k_len))
    return x, a, O.cross_visible(Tq, Tk, cu_q, cu_k, k_len)


def _run(q, k, v, dO, a, stream=None, ws=None):
    fw = M.cross_fwd(q, k, v, a, stream=stream, ws=ws)
    bw = M.cross_bwd(q, k, v, dO, fw, a, stream=stream)
    return {"O": fw["O"], "lse": fw["lse"], **bw}, fw["ws"]


def _compare(x, a, see, got, single=False):
    """single: each query sees at most one key, whose score gradient is exactly nothing."""
    f = [host64(t) for t in x]
    scale = x[0].shape[2] ** -0.5
    ref = O.attn_forward(*f[:3], see, scale, a.cap)
    ref.update(O.attn_backward(*f, see, scale, a.cap))
    lse, want = host64(got["lse"]), ref["lse"]
    assert np.array_equal(np.isneginf(lse), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.abs(lse[fin] - want[fin]).max(initial=0.0) <= LSE_ABS
    check("O", host64(got["O"]), ref["O"], REL)
    check("dV", host64(got["dV"]), ref["dV"], REL)
    for n in ("dQ", "dK"):
        if single:
            assert np.abs(host64(got[n])).max(initial=0.0) <= 1e-4, n
        else:
            check(n, host64(got[n]), ref[n], REL)
    none, unseen = ~see.any(1), ~see.any(0)
    assert not host64(got["O"])[none].any() and not host64(got["dQ"])[none].any()
    assert not host64(got["dK"])[unseen].any() and not host64(got["dV"])[unseen].any()


def _check(*shape, **kw):
    x, a, see = _make(*shape, **kw)
    got, ws = _run(*x, a)
    L.lm_workspace_check(ws)
    _compare(x, a, see, got, shape[1] == 1)
    return x, a, see, got, ws


SHAPES = [(1, 1, 1, 1, 64), (1, 2, 2, 1, 128), (1, 129, 4, 2, 128), (2, 700, 32, 8, 128), (5, 127, 5, 1, 64), (31, 300, 6, 2, 80),
          (33, 128, 20, 4, 80), (64, 1000, 8, 8, 64), (127, 65, 2, 2, 64), (129, 257, 4, 4, 96), (257, 128, 8, 2, 64),
          (300, 1, 2, 1, 8), (1, 300, 1, 1, 8), (385, 515, 6, 2, 72), (130, 1300, 16, 1, 128), (700, 90, 32, 8, 128),
          (3, 40, 300, 1, 16), (7, 1500, 1, 1, 128), (1200, 260, 7, 1, 64),
          # a key tile of many CTAs; a query tile's keys in parts; both
          (3000, 78, 4, 1, 64), (2000, 155, 4, 2, 96), (160, 4200, 20, 4, 32), (100, 2000, 4, 1, 128), (1400, 1100, 3, 1, 64)]


@pytest.mark.parametrize("Tq,Tk,hq,hk,d", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_every_query_sees_every_key(Tq, Tk, hq, hk, d, cap):
    _check(Tq, Tk, hq, hk, d, cap=cap, std=4.0 if cap else 2.0)


SEGMENTS = [  # Tq, Tk, cu_q, cu_k, k_len
    (300, 400, [0, 100, 300], [0, 250, 400], None),
    (300, 512, [0, 1, 2, 150, 300], [0, 128, 256, 384, 512], [128, 1, 77, 100]),
    (300, 400, [10, 100, 100, 280], [5, 130, 260, 390], [100, 130, 0]),      # no queries; no keys; outside
    (260, 384, [0, 60, 130, 260], [0, 128, 256, 384], [0, 128, 500]),        # a length past its places
    (257, 300, [0, 257], [40, 290], [33]),
    (40, 1290, list(range(41)), [0] + [31 + 31 * i for i in range(39)] + [1290], None),
    (3, 900, [0, 1, 2, 3], [0, 300, 600, 900], [300, 7, 250]),
    (500, 130, [0, 100, 200, 300, 400, 500], [0, 0, 30, 60, 100, 130], [0, 30, 1, 40, 30]),
    (140, 260, [140, 140], [0, 260], None),                                  # nobody sees anything
    (2600, 200, [0, 900, 901, 2600], [0, 70, 140, 200], [70, 3, 50]),        # (parts of the backward, as above)
    (2600, 150, [50, 2500], [10, 150], [100]),
    (60, 9000, [0, 20, 58], [0, 4500, 8990], [4400, 1]),
]


@pytest.mark.parametrize("Tq,Tk,cu_q,cu_k,k_len", SEGMENTS)
@pytest.mark.parametrize("hq,hk,d,cap", [(4, 2, 64, 0.0), (5, 1, 80, 3.0), (8, 8, 128, 0.0)])
def test_segments(Tq, Tk, cu_q, cu_k, k_len, hq, hk, d, cap):
    x, a, see, got, ws = _check(Tq, Tk, hq, hk, d, cap=cap, cu_q=cu_q, cu_k=cu_k, k_len=k_len)
    # what nothing sees, and what sees nothing, may hold anything
    none, unseen = (torch.from_numpy(~see.any(i)).cuda() for i in (1, 0))
    for bad in (float("nan"), float("inf")):
        y = [t.clone() for t in x]
        y[0][none], y[3][none], y[1][unseen], y[2][unseen] = bad, bad, bad, bad
        again, _ = _run(*y, a, ws=ws)
        for n in got:
            assert torch.equal(again[n], got[n]), (n, bad)


def test_one_query_of_each_of_many_sequences():
    """A batch that generates: each query its own padded states; both forms, and one after the other in a workspace."""
    for n, places in ((64, 96), (700, 12)):
        lens = [(i * 37) % places + 1 for i in range(n)]
        x, a, see, got, ws = _check(n, n * places, 16, 4, 64, cu_q=list(range(n + 1)), cu_k=list(range(0, n * places + 1, places)),
                                    k_len=lens)


def test_slices_of_a_buffer_and_head_major_layouts():
    Tq, Tk, hq, hk, d = 150, 333, 6, 2, 64
    (q, k, v, dO), a, see = _make(Tq, Tk, hq, hk, d)
    want, _ = _run(q, k, v, dO, a)
    kv = torch.cat((k, v), 1)
    wide = torch.full((Tq, hq + 3, d), float("nan"), device="cuda").bfloat16()
    wide[:, 2:2 + hq] = q
    major = dO.transpose(0, 1).contiguous().transpose(0, 1)
    for qq, kk, vv, oo in ((wide[:, 2:2 + hq], kv[:, :hk], kv[:, hk:], major),
                           (q.transpose(0, 1).contiguous().transpose(0, 1), k.transpose(0, 1).contiguous().transpose(0, 1), kv[:, hk:], dO)):
        got, _ = _run(qq, kk, vv, oo, a)
        assert all(torch.equal(got[n], want[n]) for n in want)
    one = M.cross_fwd(wide[:1, 2:2 + hq], kv[:, :hk], kv[:, hk:], a)  # (few queries, strided)
    two = M.cross_fwd(q[:1].contiguous(), k, v, a)
    assert torch.equal(one["O"], two["O"]) and torch.equal(one["lse"], two["lse"])


def test_a_layer_whose_keys_are_its_own_tokens():
    """The same as attention over packed documents that is not causal: the same arithmetic, so the same bits."""
    T, hq, hk, d = 600, 16, 8, 128  # (enough tiles for the form that has no parts)
    q, k, v, dO = _bf((T, hq, d), 1, 2.0), _bf((T, hk, d), 2), _bf((T, hk, d), 3), _bf((T, hq, d), 4)
    cu = _int32([0, 200, 450, 600])
    got, _ = _run(q, k, v, dO, M.Cross(d ** -0.5, 0.0, cu, cu))
    a = M.Attn(d ** -0.5, causal=False, cu_docs=cu)
    fw = M.attn_fwd(q, k, v, a)
    want = {"O": fw["O"], "lse": fw["lse"], **M.attn_bwd(q, k, v, dO, fw, a)}
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_nothing_on_one_side():
    q, k, v, dO = _bf((5, 4, 64), 1), _bf((0, 2, 64), 2), _bf((0, 2, 64), 3), _bf((5, 4, 64), 4)
    a = M.Cross(0.125)
    got, _ = _run(q, k, v, dO, a)
    assert not got["O"].any() and torch.isneginf(got["lse"]).all() and not got["dQ"].any() and got["dK"].shape == (0, 2, 64)
    k, v = _bf((7, 2, 64), 2), _bf((7, 2, 64), 3)
    got, _ = _run(q[:0], k, v, dO[:0], a)
    assert got["O"].shape == (0, 4, 64) and not got["dK"].any() and not got["dV"].any()


@pytest.mark.parametrize("Tq", [3, 200])
def test_a_nan_that_is_seen_and_scores_that_are_infinite(Tq):
    (q, k, v, dO), a, see = _make(Tq, 400, 4, 2, 64)
    q[1, 2, 7] = float("nan")
    fw = M.cross_fwd(q, k, v, a)
    assert fw["O"][1, 2].isnan().all() and fw["lse"][2, 1].isnan()
    keep = torch.ones(Tq, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.isfinite(fw["O"][keep]).all() and torch.isfinite(fw["lse"].T[keep]).all()


@pytest.mark.parametrize("Tq,Tk,hq,hk,d", [(1, 5000, 8, 2, 128), (260, 700, 4, 2, 64)])
def test_the_same_bits_in_a_graph_and_on_a_stream(Tq, Tk, hq, hk, d):
    n = 3 if Tq > 3 else 1
    cu_q, cu_k = [i * Tq // n for i in range(n + 1)], [i * Tk // n for i in range(n + 1)]
    x, a, see, want, _ = _check(Tq, Tk, hq, hk, d, cu_q=cu_q, cu_k=cu_k, k_len=[Tk // n - 5 * i for i in range(n)])
    ws = L.workspace(M.cross_workspace_size(Tq, Tk, hq, hk, d))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = _run(*x, a, stream=side)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = _run(*x, a, ws=ws)
    for _ in range(2):
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want)
    L.lm_workspace_check(ws)


def test_gradients_against_differences():
    (q, k, v, dO), a, see = _make(9, 37, 2, 1, 16, cap=4.0, cu_q=[0, 4, 9], cu_k=[0, 20, 37], k_len=[20, 11])
    got, _ = _run(q, k, v, dO, a)
    f = [host64(t) for t in (q, k, v)]
    up = host64(dO)
    g = np.random.default_rng(0)
    for at, n in enumerate(("dQ", "dK", "dV")):
        for _ in range(5):
            step = g.normal(size=f[at].shape)
            lo, hi = ([x + (s * step if i == at else 0) for i, x in enumerate(f)] for s in (-1e-5, 1e-5))
            slope = sum(((O.attn_forward(*y, see, 0.25, 4.0)["O"] * up).sum()) * s for y, s in ((hi, 1), (lo, -1))) / 2e-5
            d = host64(got[n])
            # (the gradient's own error is at most REL of its norm)
            assert abs((d * step).sum() - slope) <= REL * np.linalg.norm(d) * np.linalg.norm(step)


@pytest.mark.parametrize("kernel,family,Tq", [(1, 5, 300), (1, 5, 2), (2, 6, 300), (4, 7, 300)])
def test_a_starved_call_reports_a_timeout_then_recovers(kernel, family, Tq):
    (q, k, v, dO), a, see = _make(Tq, 400, 4, 2, 64)
    want, ws = _run(q, k, v, dO, a)
    fw = M.cross_fwd(q, k, v, a, ws=ws)
    assert M.call_status("attn_debug_inject", kernel, 50_000_000) == L.LM_OK
    try:
        if family == 5:
            M.cross_fwd(q, k, v, a, ws=ws)
        else:
            M.cross_bwd(q, k, v, dO, fw, a)
    finally:
        assert M.call_status("attn_debug_inject", 0, 0) == L.LM_OK
    with pytest.raises(L.LmError) as e:
        L.lm_workspace_check(ws)
    assert e.value.status == L.LM_ERR_TIMEOUT and "kernel family %d" % family in str(e.value)
    again, _ = _run(q, k, v, dO, a, ws=ws)
    L.lm_workspace_check(ws)
    assert all(torch.equal(again[n], want[n]) for n in want)


def test_offsets_past_32_bits():
    Tq, Tk, ts = 2, 3, 1 << 31
    big = torch.zeros(2 * ts + 64 * 4, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((Tk, 2, 64), (ts, 64, 1))
    v = big[128:].as_strided((Tk, 2, 64), (ts, 64, 1))
    (q, kk, vv, dO), a, see = _make(Tq, Tk, 4, 2, 64)
    k.copy_(kk)
    v.copy_(vv)
    want, _ = _run(q, kk, vv, dO, a)
    got, _ = _run(q, k, v, dO, a)
    assert all(torch.equal(got[n], want[n]) for n in want)
