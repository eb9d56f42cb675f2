"""Attention over packed documents (attn_fwd, attn_bwd) against the fp64 definition: masks, head layouts,
lengths around the 128-token tiles, strided inputs, padding that holds NaN, streams, reproducibility.

Tolerances.  Inputs are bf16, products and sums fp32.  Rounded to bf16 are, for O: P and the result; for
dV the same; for dQ and dK: P (inside delta), the score gradient and the result.  A rounding moves a
value by at most 2^-8 of itself, 2^-8 / sqrt(3) in the mean square; three independent ones give 2^-8,
and 1.5 times that, 3 x 2^-9 = 5.9e-3, bounds the relative Frobenius error.  lse is
fp32 throughout: a score's error is at most a few 2^-24 of sum |q_i k_i|, below 2e-5 at these sizes."""
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
    return (torch.randn(*shape, generator=g) * std).bfloat16()


def _int32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(T, hq, hk, d, cap=0.0, bias=False, seed=0, std=2.0, **mask):
    q, k, v, dO = _bf((T, hq, d), seed, std), _bf((T, hk, d), seed + 1), _bf((T, hk, d), seed + 2), _bf((T, hq, d), seed + 3)
    slopes = torch.tensor([2.0 ** -(1 + i % 8) for i in range(hq)]) if bias else None
    a = M.Attn(scale=d ** -0.5, cap=cap, causal=mask.get("causal", True), window=mask.get("window", 0),
               cu_docs=_int32(mask.get("cu_docs")), prefix=_int32(mask.get("prefix")),
               slopes=None if slopes is None else slopes.cuda())
    see = O.visible(T, **mask)
    f = [x.double().numpy() for x in (q, k, v)]
    sl = None if slopes is None else slopes.double().numpy()
    ref = O.attn_forward(*f, see, d ** -0.5, cap, sl)
    ref.update(O.attn_backward(*f, dO.double().numpy(), see, d ** -0.5, cap, sl))
    return [x.cuda() for x in (q, k, v, dO)], a, ref


def _run(q, k, v, dO, a, stream=None):
    fw = M.attn_fwd(q, k, v, a, stream=stream)
    bw = M.attn_bwd(q, k, v, dO, fw, a, stream=stream)
    L.lm_workspace_check(fw["ws"], stream=stream)
    return {"O": fw["O"], "lse": fw["lse"], **bw}


def _compare(got, ref, single=False):
    lse, want = host64(got["lse"]), ref["lse"]
    assert np.array_equal(np.isneginf(lse), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.abs(lse[fin] - want[fin]).max(initial=0.0) <= LSE_ABS
    check("O", host64(got["O"]), ref["O"], REL)
    check("dV", host64(got["dV"]), ref["dV"], REL)
    for n in ("dQ", "dK"):
        if single:  # every query sees one key: the score gradients are exactly nothing
            assert np.abs(host64(got[n])).max(initial=0.0) <= 1e-4, n
        else:
            check(n, host64(got[n]), ref[n], REL)


SHAPES = [(2, 2, 1, 64), (63, 4, 2, 128), (127, 2, 2, 64), (128, 4, 1, 128), (129, 4, 4, 80), (257, 8, 2, 64),
          (300, 2, 1, 8), (385, 6, 2, 96), (515, 4, 2, 128)]


@pytest.mark.parametrize("T,hq,hk,d", SHAPES)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True), (5.0, True)])
def test_causal(T, hq, hk, d, cap, bias):
    args, a, ref = _case(T, hq, hk, d, cap, bias, seed=T)
    _compare(_run(*args, a), ref)


MASKS = {
    "full": (200, dict(causal=False)),
    "full window": (300, dict(causal=False, window=70)),
    "window": (400, dict(window=33)),
    "window longer than T": (140, dict(window=4096)),
    "documents": (520, dict(cu_docs=[0, 1, 1, 130, 131, 259, 400, 520])),
    "documents, padded at both ends": (520, dict(cu_docs=[5, 100, 390, 401])),
    "all padding but one": (300, dict(cu_docs=[131, 133])),
    "prefix": (400, dict(cu_docs=[0, 150, 400], prefix=[150, 70])),
    "prefix longer than its document": (260, dict(cu_docs=[0, 3, 140, 260], prefix=[9, 1000, 0])),
    "prefix, window": (390, dict(cu_docs=[0, 260, 380], prefix=[200, 60], window=90)),
    "full documents": (400, dict(causal=False, cu_docs=[0, 128, 129, 384])),
    "tiny documents": (260, dict(cu_docs=list(range(0, 257, 4)))),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", list(MASKS))
def test_masks(name, d):
    T, mask = MASKS[name]
    for cap, bias in ((0.0, False), (4.0, True)):
        m = dict(mask)
        if "prefix" in m:  # (a prefix is clamped to its document)
            m["prefix"] = [min(p, b - a) for p, a, b in zip(m["prefix"], m["cu_docs"], m["cu_docs"][1:])]
        args, a, ref = _case(T, 4, 2, d, cap, bias, seed=T + d, **m)
        a.prefix = _int32(mask.get("prefix"))
        _compare(_run(*args, a), ref)


@pytest.mark.parametrize("T,mask", [(1, {}), (130, dict(window=1)), (140, dict(cu_docs=list(range(0, 141))))])
def test_every_token_sees_itself_alone(T, mask):
    args, a, ref = _case(T, 4, 2, 64, seed=9, **mask)
    _compare(_run(*args, a), ref, single=True)


def test_nothing_is_seen():
    args, a, ref = _case(200, 4, 2, 64, seed=4, cu_docs=[0, 0])
    got = _run(*args, a)
    assert torch.all(got["lse"] == -float("inf"))
    for n in ("O", "dQ", "dK", "dV"):
        assert torch.all(got[n] == 0), n


def test_no_tokens():
    q, k = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    a = M.Attn(scale=1.0)
    fw = M.attn_fwd(q, k, k, a)
    bw = M.attn_bwd(q, k, k, q, fw, a)
    assert fw["O"].shape == (0, 4, 64) and bw["dK"].shape == (0, 2, 64)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, True)])
def test_padding_may_hold_anything(cap, bias):
    (q, k, v, dO), a, ref = _case(300, 4, 2, 64, cap, bias, seed=21, cu_docs=[6, 150, 290])
    clean = _run(q, k, v, dO, a)
    for x in (q, k, v, dO):
        x[:6] = float("nan")
        x[290:295] = float("inf")
        x[295:] = float("nan")
    got = _run(q, k, v, dO, a)
    _compare(got, ref)
    for n in clean:
        assert torch.equal(clean[n], got[n]), n


def test_strided_inputs():
    (q, k, v, dO), a, ref = _case(270, 4, 2, 80, 3.0, seed=31, cu_docs=[0, 100, 270])
    want = _run(q, k, v, dO, a)
    qkv = torch.full((270, 4 + 2 + 2, 80), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :4], qkv[:, 4:6], qkv[:, 6:] = q, k, v                                # one fused buffer
    major = dO.transpose(0, 1).contiguous().transpose(0, 1)                      # head-major
    wide = torch.full((270, 2, 104), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, :80] = v                                                          # a gap after each head
    gap = torch.full((270, 2 * 80 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    gap[:, 8:] = k.reshape(270, 160)                                             # a gap after each token, base 16 bytes on
    for args in ((qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], major), (q, gap[:, 8:].unflatten(1, (2, 80)), wide[:, :, :80], dO)):
        got = _run(*args, a)
        for n in want:
            assert torch.equal(want[n], got[n]), n


@pytest.mark.parametrize("T,d", [(700, 128), (513, 64)])
def test_same_bits_again_and_on_a_side_stream(T, d):
    args, a, _ = _case(T, 4, 1, d, 6.0, True, seed=17, cu_docs=[0, T // 3, T], prefix=[10, 90])
    want = _run(*args, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, None):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            got = _run(*args, a, stream=stream)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(want[n], got[n]), n


def test_large_scores_stay_finite():
    """Scores in the thousands: one key takes all of each row's weight, and nothing overflows."""
    (q, k, v, dO), a, ref = _case(200, 2, 1, 64, seed=51, std=300.0)
    got = _run(q, k, v, dO, a)
    check("O", host64(got["O"]), ref["O"], REL)
    for n in ("dQ", "dK", "dV"):
        assert torch.isfinite(got[n].float()).all(), n


def test_gradients_against_differences():
    """Directional differences of the forward itself: its O moves by what dQ, dK, dV say."""
    (q, k, v, dO), a, _ = _case(192, 4, 2, 64, 8.0, True, seed=61, cu_docs=[0, 70, 192])
    got = _run(q, k, v, dO, a)

    def f(q, k, v):
        return (M.attn_fwd(q, k, v, a)["O"].double() * dO.double()).sum().item()

    for name, x, at in (("dQ", q, 0), ("dK", k, 1), ("dV", v, 2)):
        step = _bf(tuple(x.shape), 70 + at, 1.0).cuda()
        step = torch.sign(got[name].float()) * step.abs().float()          # a direction in which f rises steadily
        rate = []
        for h in (0.125, 0.0625):
            ins = [[q, k, v] for _ in range(2)]
            ins[0][at], ins[1][at] = (x.float() + h * step).bfloat16(), (x.float() - h * step).bfloat16()
            taken = (ins[0][at].float() - ins[1][at].float()).double()     # what rounding left of the step
            rate.append((f(*ins[0]) - f(*ins[1])) / (got[name].double() * taken).sum().item())
        # two steps take the third-order term out; the fifth-order one and the bf16 roundings of the forwards
        # (which weigh more in a smaller step) leave a few per cent
        assert abs((4 * rate[1] - rate[0]) / 3 - 1) <= 0.05, (name, rate)


def test_offsets_past_32_bits():
    """128 heads of 128 over 140000 tokens: q, O, dO and dQ have 2.3e9 elements each.  A window of 40 keeps
    the work small; rows from both ends are checked against the definition on their own neighbourhood."""
    T, hq, hk, d, W = 140000, 128, 2, 128, 40
    assert T * hq * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, dO = (torch.randn(T, h, d, generator=g, device="cuda", dtype=torch.bfloat16) for h in (hq, hk, hk, hq))
    a = M.Attn(scale=d ** -0.5, window=W)
    got = _run(q, k, v, dO, a)
    n = 200
    for s in (0, T - n):
        sl = slice(s, s + n)
        see = O.visible(n, window=W)
        for h, gk in ((0, 0), (127, 1)):
            f = [x[sl, i:i + 1].double().cpu().numpy() for x, i in ((q, h), (k, gk), (v, gk))]
            ref = O.attn_forward(*f, see, d ** -0.5)
            ref.update(O.attn_backward(*f, dO[sl, h:h + 1].double().cpu().numpy(), see, d ** -0.5))
            inner = slice(0 if s == 0 else W, n)  # rows whose keys are all in the slice
            check("O", host64(got["O"][sl, h])[inner], ref["O"][inner, 0], REL)
            check("dQ", host64(got["dQ"][sl, h])[inner], ref["dQ"][inner, 0], REL)
    del q, dO, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,hq,hk,d", [(2600, 8, 8, 64), (1300, 16, 8, 128), (520, 8, 2, 128), (260, 5, 1, 128), (700, 6, 2, 40)])
@pytest.mark.parametrize("docs", [False, True])
def test_key_tiles_of_one_two_and_four_ctas(T, hq, hk, d, docs):
    """dK and dV where there are more key tiles than SMs, fewer, and far fewer (their sums then meet from two
    or four CTAs), with documents whose key tiles are taken out of order."""
    mask = dict(cu_docs=[0, 3, 3, T // 7, T // 7 + 1, T // 2, T - 9]) if docs else {}
    args, a, ref = _case(T, hq, hk, d, seed=11, **mask)
    got, again = _run(*args, a), _run(*args, a)
    _compare(got, ref)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("cap", [2.0 ** -14, 0.3, 1000.0])
def test_caps_far_from_the_scores(cap):
    """Scores all but cut off, and all but left alone.  1 / (1 + e) near 1/2 is off by 2^-24.5 (the exponential,
    2 ulp, of which a quarter counts), 2^-25 (the sum's rounding) and 2^-24 (the reciprocal, 1 ulp), times 2 cap;
    the maximum and lse are rounded at the size of the cap, 2^-24 each: together below 2^-21.5 cap."""
    args, a, ref = _case(200, 2, 1, 64, cap, seed=31)
    got = _run(*args, a)
    lse, want = host64(got["lse"]), ref["lse"]
    assert np.abs(lse - want).max() <= LSE_ABS + cap * 2.0 ** -21.5
    for n in ("O", "dV", "dQ", "dK"):
        if cap < 1e-3 and n in ("dQ", "dK"):  # (du/dz underflows nearly everywhere)
            assert np.isfinite(host64(got[n])).all()
        else:
            check(n, host64(got[n]), ref[n], REL)
