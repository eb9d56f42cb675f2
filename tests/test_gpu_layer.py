"""The layer operators at work together and with the device: a LoRA decoder layer over packed documents
(examples/packed_layer.py) against the fp64 definitions chained the same way, calls on a stream of
their own, and the attention kernels' bounded waits made to run out.

Tolerances of the chained step.  Every tensor between two operators is rounded to bf16, as are the rank-r
products, the attention weights and their gradients: 15 roundings on the longest path forward, 12
backward, each 2^-8 / sqrt(3) in the mean square at most, together 1.2e-2; twice that, 2.5e-2, for what
grows on the way (a residual sum's rounding is relative to the sum, not to the branch).  The loss
averages over 200 targets or more errors of 1.2e-2 at logits of size 1: 1e-2 is far outside."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O
from oracle import lora as OL

from gpu_util import check, host64

pytestmark = pytest.mark.gpu

STEP_REL = 2.5e-2
WAIT_NS = 50_000_000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "packed_layer.py")
    spec = importlib.util.spec_from_file_location("packed_layer", path)
    mod = importlib.util.module_from_spec(spec)
    sys.modules["packed_layer"] = mod  # (its dataclass looks its module up)
    spec.loader.exec_module(mod)
    return mod


# ------------------------------------------------------------------------------------ the step
def _reference(layer, tokens, targets, cu):
    s, p = layer.s, {n: host64(t) for n, t in layer.params.items()}
    W = {n: host64(lo.W) for n, lo in layer.lora.items()}

    def lora(names, keys):
        q = {}
        for n, k in zip(names, keys):
            q["W" + k], q["A" + k], q["B" + k], q["s" + k] = W[n], p["A_" + n], p["B_" + n], layer.lora[n].s
        return q

    h0, head, tgt = host64(layer.embed[tokens]), host64(layer.head), targets.cpu().numpy()
    sl, T, eps = host64(layer.slopes), h0.shape[0], M.AddNorm().eps
    see = O.visible(T, cu_docs=cu.cpu().tolist())
    n1 = O.addnorm_forward(h0, None, p["w_attn"], eps=eps)
    pq, pm = lora(("q", "k", "v"), "qkv"), lora(("gate", "up", "down"), "gud")
    qkv = OL.qkv_forward(n1["x"], pq)
    q, k, v = (qkv[x].reshape(T, -1, s.head) for x in "QKV")
    a = O.attn_forward(q, k, v, see, s.head ** -0.5, 0.0, sl)["O"].reshape(T, -1)
    po = (W["o"], p["A_o"], p["B_o"], layer.lora["o"].s)
    o, _ = OL.lora_w_forward(a, *po)
    n2 = O.addnorm_forward(h0, o, p["w_mlp"], eps=eps)
    y = OL.mlp_forward(n2["x"], pm)["y"]
    n3 = O.addnorm_forward(n2["h"], y, p["w_head"], eps=eps)
    logits = n3["x"] @ head.T
    has = tgt >= 0
    loss = -O.logprob_forward(logits, tgt)["logp"].sum() / has.sum()
    g = {}
    dx3 = O.logprob_backward(logits, tgt, np.full(T, -1.0 / has.sum())) @ head
    b3 = O.addnorm_backward(n2["h"], y, None, dx3, p["w_head"], eps=eps)
    bm = OL.mlp_backward(n2["x"], b3["dy"], pm)
    b2 = O.addnorm_backward(h0, o, b3["dh"], bm["dX"], p["w_mlp"], eps=eps)
    bo = OL.lora_w_backward(a, b2["dy"], *po)
    g["A_o"], g["B_o"] = bo["dA"], bo["dB"]
    ba = O.attn_backward(q, k, v, bo["dX"].reshape(T, -1, s.head), see, s.head ** -0.5, 0.0, sl)
    bq = OL.qkv_backward(n1["x"], *(ba["d" + x].reshape(T, -1) for x in "QKV"), pq)
    g["w_attn"] = O.addnorm_backward(h0, None, b2["dh"], bq["dX"], p["w_attn"], eps=eps)["dw_in"]
    g["w_mlp"], g["w_head"] = b2["dw_in"], b3["dw_in"]
    for part, names, keys in ((bm, ("gate", "up", "down"), "gud"), (bq, ("q", "k", "v"), "qkv")):
        for n, k in zip(names, keys):
            g["A_" + n], g["B_" + n] = part["dA" + k], part["dB" + k]
    return loss, g


def test_a_packed_lora_layer_against_the_chained_definitions(example):
    s = example.Sizes(T=300, d=256, n=704, hq=4, hk=2, head=64, V=1000, r=8)
    layer = example.PackedLayer(s, seed=3, b_std=0.02)
    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(s.V, (s.T,), generator=g).cuda()
    cu = torch.tensor([0, 1, 3, 130, 130, 287], dtype=torch.int32, device="cuda")  # 13 tokens of padding
    targets = torch.randint(s.V, (s.T,), generator=g).cuda()
    targets[[0, 2, 129]] = -1
    targets[286:] = -1
    want, ref = _reference(layer, tokens, targets, cu)
    f = layer.forward(tokens, cu)
    loss = float(layer.loss(f, targets))
    got = layer.backward(f, targets)
    for ws in (f["qkv"]["ws"], f["att"]["ws"], f["o"]["ws"], f["mlp"]["ws"]):
        L.lm_workspace_check(ws)
    assert abs(loss - want) <= 1e-2, (loss, want)
    assert set(got) == set(ref) == set(layer.params)
    for n in ref:
        check(n, host64(got[n]), ref[n], STEP_REL, 2 * STEP_REL)


def test_the_example_learns(example):
    s = example.Sizes(T=700, d=256, n=512, hq=4, hk=1, head=128, V=500)
    tokens, targets, cu = example.packed_documents(s.T, s.V)
    losses = example.train(example.PackedLayer(s), tokens, targets, cu, 8, 1e-2, log=lambda line: None)
    assert np.isfinite(losses).all() and losses[-1] < losses[0] - 0.1, losses
    top = example.continuations(example.PackedLayer(s), tokens, cu, 1, k=3)
    assert top["top_ids"].shape == (1, 3) and (top["top_logp"][0, 0] >= top["top_logp"][0, 1])


# ------------------------------------------------------------------------------------ streams
def _attn_case(T=300, hq=4, hk=2, d=64):
    g = torch.Generator().manual_seed(1)
    q, k, v, dO = (torch.randn(T, h, d, generator=g).bfloat16().cuda() for h in (hq, hk, hk, hq))
    return q, k, v, dO, M.Attn(scale=0.125, cu_docs=torch.tensor([0, 100, T], dtype=torch.int32, device="cuda"))


def test_a_stream_given_by_argument():
    """The current stream is busy; the call's own stream is not, and what it allocates and zeroes is ordered
    there."""
    q, k, v, dO, a = _attn_case()
    g = torch.Generator().manual_seed(2)
    h, y, dx = (torch.randn(300, 256, generator=g).bfloat16().cuda() for _ in range(3))
    n = M.AddNorm(w_in=torch.ones(256, device="cuda"))
    t = torch.randint(256, (300,), generator=g).cuda()

    def run(**kw):
        fw = M.attn_fwd(q, k, v, a, **kw)
        bw = M.attn_bwd(q, k, v, dO, fw, a, **kw)
        an = M.addnorm_fwd(h, y, n, **kw)
        ab = M.addnorm_bwd(h, y, None, dx, an, n, **kw)
        lp = M.logprob_fwd(h, t, **kw)
        lb = M.logprob_bwd(h, t, lp, lp["lse"], **kw)
        return [fw["O"], fw["lse"], bw["dQ"], bw["dK"], bw["dV"], an["x"], ab["dh"], ab["dw_in"], lp["logp"],
                lb["dlogits"]], fw["ws"]

    want, _ = run()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        for _ in range(20):
            big @ big
        got, ws = run(stream=stream)
        L.lm_workspace_check(ws, stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()


def test_a_captured_step_replays_the_same_bits():
    q, k, v, dO, a = _attn_case()
    h, dx = (torch.randn(300, 256, device="cuda").bfloat16() for _ in range(2))
    n = M.AddNorm(w_in=torch.ones(256, device="cuda"))
    t = torch.randint(256, (300,), device="cuda")
    ws, wn = L.workspace(M.attn_workspace_size(300, 4, 2, 64)), L.workspace(M.addnorm_workspace_size(300, 256))

    def step():
        fw = M.attn_fwd(q, k, v, a, ws=ws)
        out = [fw["O"], fw["lse"], *M.attn_bwd(q, k, v, dO, fw, a).values()]
        an = M.addnorm_fwd(h, fw["O"].view(300, 256), n)
        ab = M.addnorm_bwd(h, fw["O"].view(300, 256), None, dx, an, n, ws=wn)
        lp = M.logprob_fwd(an["x"], t, k=4)
        out += [an["x"], ab["dh"], ab["dy"], ab["dw_in"], lp["logp"], lp["top_ids"]]
        return out + [M.logprob_bwd(an["x"], t, lp, lp["entropy"])["dlogits"]]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    L.lm_workspace_check(ws)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------------------------ bounded waits
@pytest.mark.parametrize("kernel,family", [(1, 5), (2, 6), (4, 7)])
@pytest.mark.parametrize("T,hq,hk,d", [(300, 4, 2, 64), (520, 8, 1, 128)])  # (the second: four CTAs a key tile)
def test_starved_attention_reports_timeout_then_recovers(kernel, family, T, hq, hk, d):
    q, k, v, dO, a = _attn_case(T, hq, hk, d)
    ws = L.workspace(M.attn_workspace_size(T, hq, hk, d))
    fw = M.attn_fwd(q, k, v, a, ws=ws)
    want = M.attn_bwd(q, k, v, dO, fw, a)
    L.lm_workspace_check(ws)
    assert M.call_status("attn_debug_inject", kernel, WAIT_NS) == L.LM_OK
    try:
        if family == 5:
            M.attn_fwd(q, k, v, a, ws=ws)
        else:
            M.attn_bwd(q, k, v, dO, fw, a)
    finally:
        assert M.call_status("attn_debug_inject", 0, 0) == L.LM_OK
    with pytest.raises(L.LmError) as ei:
        L.lm_workspace_check(ws)
    assert ei.value.status == L.LM_ERR_TIMEOUT and "kernel family %d" % family in str(ei.value)
    L.lm_workspace_check(ws)  # the check cleared the word
    again = M.attn_fwd(q, k, v, a, ws=ws)
    got = M.attn_bwd(q, k, v, dO, again, a)
    L.lm_workspace_check(ws)
    assert torch.equal(again["O"], fw["O"]) and all(torch.equal(got[n], want[n]) for n in want)
