"""Many calls of cross attention over documents with padded states, in all forms of the forward and beside each other: no
wait runs out, and every call has the same bits.  (What orders the ring's fills is modelled in test_attn_ring_host.py.)"""
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


@pytest.mark.parametrize("Tq,Tk,docs,hq,hk,d", [(64, 64 * 300, 64, 32, 8, 128), (40, 40 * 500, 40, 8, 8, 64), (3, 9000, 3, 4, 2, 128),
                                                (1500, 6000, 5, 16, 4, 128), (1300, 9000, 9, 20, 4, 64)])
def test_many_calls_beside_each_other(Tq, Tk, docs, hq, hk, d):
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((Tq, hq, d), (Tk, hk, d), (Tk, hk, d)))
    of = lambda n: torch.tensor([i * n // docs for i in range(docs + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    used = torch.tensor([max(1, Tk // docs - 37 * i % (Tk // docs)) for i in range(docs)], dtype=torch.int32, device="cuda")
    a = M.Cross(d ** -0.5, 0.0, of(Tq), of(Tk), used)
    want = M.cross_fwd(q, k, v, a)
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [L.workspace(M.cross_workspace_size(Tq, Tk, hq, hk, d)) for _ in streams]
    outs = [(torch.empty_like(want["O"]), torch.empty_like(want["lse"])) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(20):
            for s, ws, (o, lse) in zip(streams, spaces, outs):
                M.cross_fwd(q, k, v, a, train=False, O=o, lse=lse, ws=ws, stream=s)
        torch.cuda.synchronize()
        for ws, (o, lse) in zip(spaces, outs):
            L.lm_workspace_check(ws)
            assert torch.equal(o, want["O"]) and torch.equal(lse, want["lse"])
            o.zero_()
            lse.zero_()
        torch.cuda.synchronize()
