"""Cross attention's backward where documents end with whole tiles and keys of no document lie behind them: those keys' tiles
have no queries, and ask for none; their gradients are zeros, whatever they hold.  (Tolerances as in test_gpu_cross.py.)"""
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


@pytest.mark.parametrize("Tq,cu_q,Tk,cu_k", [(128, [0, 128], 900, [0, 200]), (256, [0, 100, 256], 1024, [0, 128, 256]),
                                             (2560, [0, 1300, 2560], 400, [0, 60, 128])])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (8, 8, 128)])
def test_key_tiles_behind_the_last_document(Tq, cu_q, Tk, cu_k, hq, hk, d):
    g = torch.Generator().manual_seed(1)
    q, k, v, dO = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((Tq, hq, d), (Tk, hk, d), (Tk, hk, d), (Tq, hq, d)))
    k[cu_k[-1]:], v[cu_k[-1]:] = float("nan"), float("inf")
    a = M.Cross(d ** -0.5, 0.0, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu_q, cu_k)))
    fw = M.cross_fwd(q, k, v, a)
    got = M.cross_bwd(q, k, v, dO, fw, a)
    L.lm_workspace_check(fw["ws"])
    n, f = cu_k[-1], [host64(t) for t in (q, k[:cu_k[-1]], v[:cu_k[-1]])]
    ref = O.attn_backward(*f, host64(dO), O.cross_visible(Tq, n, cu_q, cu_k), d ** -0.5)
    for name in ("dK", "dV"):
        assert not got[name][n:].any()
        check(name, host64(got[name][:n]), ref[name], REL)
    check("dQ", host64(got["dQ"]), ref["dQ"], REL)
