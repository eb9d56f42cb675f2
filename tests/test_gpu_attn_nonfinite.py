"""NaN and infinities inside a document (attn_fwd, attn_bwd): what the definition makes NaN is NaN, never a
finite number or a zero, and what no such value reaches has the bits of a clean run.

By the definition a query that sees a NaN key, or is one, has NaN weights: O, lse and dQ of it, and dK and dV
of every key that it sees.  A NaN value leaves the weights alone: O and dQ of the queries that see it, and dK of
the keys that those see, are NaN; lse and dV are not.  Rows that see none of it are compared in documents that
have no token in the value's tile of 128, and in its own where no product of nothing with NaN can reach them."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import check, host64

pytestmark = pytest.mark.gpu

CU, T, HQ, HK = [0, 256, 640, 700], 700, 4, 2  # the poisoned document has tiles 2, 3, 4 to itself


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _bf(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16().cuda()


def _run(q, k, v, dO, a):
    fw = M.attn_fwd(q, k, v, a)
    bw = M.attn_bwd(q, k, v, dO, fw, a)
    L.lm_workspace_check(fw["ws"])
    return {"O": fw["O"], "lse": fw["lse"].T, **bw}  # (all by token first)


def _attn(d, see, cap, bias, cu=CU):
    pre = see.get("prefix")
    return M.Attn(scale=d ** -0.5, cap=cap, causal=see.get("causal", True), window=see.get("window", 0),
                  cu_docs=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                  prefix=None if pre is None else torch.tensor(pre, dtype=torch.int32, device="cuda"),
                  slopes=torch.tensor([2.0 ** -(1 + i) for i in range(HQ)], device="cuda") if bias else None)


def _reached(which, at, see):
    """Truth values by the definition, (token, head), of what a NaN token `at` of head 0 makes NaN."""
    n = HQ // HK
    rows = np.zeros((T, HQ), dtype=bool)
    if which == "q":
        rows[at, 0] = see[at].any()
    else:
        rows[:, :n] = see[:, at][:, None]
    keys = np.zeros((T, HK), dtype=bool)
    for h in range(HQ):
        keys[:, h // n] |= see[rows[:, h]].any(axis=0)
    none_rows, none_keys = np.zeros_like(rows), np.zeros_like(keys)
    return {"O": rows, "dQ": rows, "dK": keys, "lse": none_rows if which == "v" else rows,
            "dV": none_keys if which == "v" else keys}


# 0 x NaN reaches rows of the document that see nothing of it: a NaN row on the right of the product
SPREADS = {"q": ("dK",), "k": ("dQ",), "v": ("O", "dQ", "dK")}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("mask", [dict(), dict(causal=False), dict(window=90), dict(prefix=[9, 150, 0])], ids=str)
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_nan_inside_a_document(which, mask, cap, bias, d):
    args = dict(zip(("q", "k", "v", "dO"), (_bf((T, HQ, d), 1, 2.0), _bf((T, HK, d), 2), _bf((T, HK, d), 3), _bf((T, HQ, d), 4))))
    a = _attn(d, mask, cap, bias)
    clean = _run(**args, a=a)
    see = O.visible(T, cu_docs=CU, **mask)
    inside = np.zeros(T, dtype=bool)
    inside[CU[1]:CU[2]] = True
    for at in (CU[1] + 3, CU[1] + 200, CU[2] - 1):  # the document's first, a middle and its last tile
        bad = dict(args)
        bad[which] = args[which].clone()
        bad[which][at, 0] = float("nan")
        got = _run(**bad, a=a)
        for n, hit in _reached(which, at, see).items():
            x, c = got[n].float().cpu().numpy(), clean[n].float().cpu().numpy()
            assert np.isnan(x[hit]).all(), (n, at)
            same = ~hit
            if n in SPREADS[which]:
                same &= ~inside[:, None]
            assert np.array_equal(x[same], c[same]), (n, at)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("at", [2, 70, 199])
def test_infinite_scores(at, bias):
    """One infinite element of one key: a score of +inf has no softmax (NaN), one of -inf has no weight."""
    d, n = 64, 200
    q, k, v = _bf((n, HQ, d), 11, 2.0), _bf((n, HK, d), 12), _bf((n, HK, d), 13)
    k[at, 0, 5] = float("inf")
    a = _attn(d, {}, 0.0, bias, cu=[0, n])
    fw = M.attn_fwd(q, k, v, a)
    L.lm_workspace_check(fw["ws"])
    see = O.visible(n)
    got, lse = host64(fw["O"]), host64(fw["lse"])
    sl = None if a.slopes is None else a.slopes.double().cpu().numpy()
    k0 = k.clone()
    k0[at, 0] = 0
    for h in range(HQ):
        up = see[:, at] & (host64(q)[:, h, 5] > 0) & (h < HQ // HK)
        assert np.isnan(got[up, h]).all() and np.isnan(lse[h, up]).all(), h
        hide = see.copy()
        if h < HQ // HK:
            hide[:, at] = False
        f = [host64(x)[:, i:i + 1] for x, i in ((q, h), (k0, h * HK // HQ), (v, h * HK // HQ))]
        ref = O.attn_forward(*f, hide, d ** -0.5, 0.0, None if sl is None else sl[h:h + 1])
        check("O", got[~up, h], ref["O"][~up, 0], 3 * 2.0 ** -9)
        fin = ~up & np.isfinite(ref["lse"][0])  # (a first token whose only key has -inf sees nothing that counts)
        assert np.array_equal(np.isneginf(lse[h, ~up]), np.isneginf(ref["lse"][0, ~up]))
        assert np.abs(lse[h, fin] - ref["lse"][0, fin]).max() <= 2e-5
