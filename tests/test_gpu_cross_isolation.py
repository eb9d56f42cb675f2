"""What a document's infinities and NaN do to others in cross attention.  Forward: nothing, in any form, wherever the documents
lie; the document's own results are not finite where its values say so, and right elsewhere.  Backward: nothing to
documents that share no 128 queries and no 128 keys (from a multiple of 128 on) with it.

Tolerances as in test_gpu_cross.py: P and the result are rounded to bf16, 3 x 2^-9 of the norm.  With the bits of O_lo, of
rows that were formed again (in fp32 throughout): those hold a value to 2^-16 of itself, the rest is below 2^-17."""
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _even(n, parts):
    return [n * i // parts for i in range(parts + 1)]


def _inputs(Tq, Tk, hq, hk, d):
    g = torch.Generator().manual_seed(7)
    return [(torch.randn(*s, generator=g) * f).bfloat16().cuda() for s, f in
            (((Tq, hq, d), 2), ((Tk, hk, d), 1), ((Tk, hk, d), 1), ((Tq, hq, d), 1))]


FORMS = [  # Tq, Tk, documents, hq, hk, d, cap
    (64, 64 * 300, 64, 32, 8, 128, 0.0),   # a batch that generates: the keys in parts
    (12, 12 * 900, 12, 4, 2, 64, 3.0),
    (30, 100, 10, 8, 2, 80, 0.0),          # one tile of keys: no parts
    (9, 120, 3, 4, 4, 64, 0.0),
    (700, 900, 6, 16, 4, 128, 0.0),        # a tile of queries an item, and two
    (1500, 1400, 7, 20, 4, 72, 5.0),
    (3000, 3000, 3, 8, 8, 64, 0.0),
]


@pytest.mark.parametrize("Tq,Tk,docs,hq,hk,d,cap", FORMS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("what", ["values", "one value", "keys", "queries"])
def test_a_document_does_not_change_the_others_results(Tq, Tk, docs, hq, hk, d, cap, bad, what):
    q, k, v, _ = _inputs(Tq, Tk, hq, hk, d)
    cu_q, cu_k = _even(Tq, docs), _even(Tk, docs)
    used = [max(1, cu_k[i + 1] - cu_k[i] - 3 * i % 5) for i in range(docs)]
    a = M.Cross(d ** -0.5, cap, _int32(cu_q), _int32(cu_k), _int32(used))
    see = O.cross_visible(Tq, Tk, cu_q, cu_k, used)
    ref = O.attn_forward(*(host64(t) for t in (q, k, v)), see, d ** -0.5, cap)
    clean = M.cross_fwd(q, k, v, a)
    sick = docs // 2
    q0, q1, k0 = cu_q[sick], cu_q[sick + 1], cu_k[sick]
    at = k0 + used[sick] // 2
    if what == "values":
        v[k0:k0 + used[sick]] = bad
    elif what == "one value":
        v[at, 0, 3] = bad
    elif what == "keys":
        k[at, :, 5] = bad
    else:
        q[q0:q1, :, 1] = bad
    got = M.cross_fwd(q, k, v, a)
    L.lm_workspace_check(got["ws"])
    own = torch.zeros(Tq, dtype=torch.bool, device="cuda")
    own[q0:q1] = True
    assert torch.equal(got["lse"][:, ~own], clean["lse"][:, ~own])
    rest = (~own).cpu().numpy()
    check("O", host64(got["O"])[rest], ref["O"][rest], REL)
    more = (got["O"].view(torch.int16).to(torch.int32) << 16) + got["O_lo"][..., :d].to(torch.int32) * 256
    check("O and its low bits", host64(more.view(torch.float32))[rest], ref["O"][rest], REL)
    again = (got["O"] != clean["O"]).any(-1)[~own].cpu().numpy()  # (rows that were formed again, about)
    if again.any():
        check("rows formed again", host64(more.view(torch.float32))[rest][again], ref["O"][rest][again], 2.0 ** -15, 2.0 ** -15)
    o = got["O"][own]
    if what == "one value":
        first = torch.zeros(hq, d, dtype=torch.bool, device="cuda")
        first[:hq // hk, 3] = True
        assert not torch.isfinite(o[:, first]).any() and torch.isfinite(o[:, ~first]).all()
        assert torch.equal(got["lse"], clean["lse"])
        mine, others = own.cpu().numpy(), ~first.cpu().numpy()
        check("the other dims", host64(got["O"])[mine][:, others], ref["O"][mine][:, others], REL)
    elif what == "values":
        assert not torch.isfinite(o).any()


@pytest.mark.parametrize("cap", [0.0, 4.0])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_of_documents_that_share_no_tile(bad, cap):
    hq, hk, d = 8, 2, 64
    cu_q, cu_k = [0, 200, 384, 600], [0, 300, 512, 700]  # (the third begins with tiles of its own, of queries and of keys)
    x = _inputs(600, 700, hq, hk, d)
    a = M.Cross(d ** -0.5, cap, _int32(cu_q), _int32(cu_k))

    def run():
        fw = M.cross_fwd(*x[:3], a)
        got = M.cross_bwd(*x, fw, a)
        L.lm_workspace_check(fw["ws"])
        return {**got, "O": fw["O"]}

    want = run()
    for t in x:
        t[5, 0, 7] = bad
    got = run()
    for n, at in (("O", 384), ("dQ", 384), ("dK", 512), ("dV", 512)):
        assert torch.equal(got[n][at:], want[n][at:]) and torch.isfinite(got[n][at:]).all(), n
