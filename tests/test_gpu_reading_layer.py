"""The operators of a layer that reads images at work together (examples/reading_layer.py): norm and rotation of heads
by three axes, attention to padded encoder states, the loss against a teacher, next to the projections, the other
attention and the norms, against the fp64 definitions chained the same way; the step captured in a CUDA graph beside an
eager one; and the example's run.

Tolerances of the chained step.  Every tensor between two operators is rounded to bf16, as are the rank-r products, the
attention weights and their gradients: 22 roundings on the longest path forward, 19 backward, each 2^-8 / sqrt(3) in the
mean square at most, together 2^-8 sqrt(41 / 3) = 1.4e-2; twice that, 2.9e-2, for what grows on the way (a residual
sum's rounding is relative to the sum, not to the branch).  The loss averages over some hundred targets errors of
1.4e-2 at logits of size 1: 1e-2 is far outside."""
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

STEP_REL = 2.9e-2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "reading_layer.py")
    spec = importlib.util.spec_from_file_location("reading_layer", path)
    mod = importlib.util.module_from_spec(spec)
    sys.modules["reading_layer"] = mod  # (its dataclasses look their module up)
    spec.loader.exec_module(mod)
    return mod


def _reference(layer, b):
    s, p = layer.s, {n: host64(t) for n, t in layer.params.items()}
    W = {n: host64(lo.W) for n, lo in layer.lora.items()}

    def keyed(names, keys):
        q = {}
        for n, k in zip(names, keys):
            q["W" + k], q["A" + k], q["B" + k], q["s" + k] = W[n], p["A_" + n], p["B_" + n], layer.lora[n].s
        return q

    one = lambda n: (W[n], p["A_" + n], p["B_" + n], layer.lora[n].s)  # noqa: E731
    heads = lambda x: x.reshape(x.shape[0], -1, s.head)  # noqa: E731
    flat = lambda x: x.reshape(x.shape[0], -1)  # noqa: E731
    np_ = lambda t: t.cpu().numpy()  # noqa: E731
    eps, sc = M.AddNorm().eps, s.head ** -0.5
    head, tgt, T = host64(layer.head), np_(b.targets), s.T
    see = O.visible(T, cu_docs=np_(b.cu).tolist())
    csee = O.cross_visible(T, s.S, np_(b.cu).tolist(), np_(b.cu_states).tolist(), np_(b.used).tolist())
    rot = dict(angles=O.qkrope_angles(T, np_(layer.inv_freq), np_(b.pos), np_(layer.axis)), norm=True, eps=M.QkRope().eps)
    nrm = dict(norm=True, eps=M.QkRope().eps)
    h0, st = host64(layer.embed[b.tokens]), host64(b.states)
    n1 = O.addnorm_forward(h0, None, p["w_attn"], eps=eps)
    pq, pm = keyed(("q", "k", "v"), "qkv"), keyed(("gate", "up", "down"), "gud")
    qkv = OL.qkv_forward(n1["x"], pq)
    q0, k0, v = (heads(qkv[x]) for x in "QKV")
    q, k = O.qkrope_forward(q0, w=p["w_q"], **rot), O.qkrope_forward(k0, w=p["w_k"], **rot)
    a = flat(O.attn_forward(q, k, v, see, sc)["O"])
    o, _ = OL.lora_w_forward(a, *one("o"))
    n2 = O.addnorm_forward(h0, o, p["w_cross"], eps=eps)
    cq, ck, cv = (heads(OL.lora_w_forward(x, *one(n))[0]) for x, n in ((n2["x"], "cq"), (st, "ck"), (st, "cv")))
    cqn, ckn = O.qkrope_forward(cq, w=p["w_cq"], **nrm), O.qkrope_forward(ck, w=p["w_ck"], **nrm)
    c = flat(O.attn_forward(cqn, ckn, cv, csee, sc)["O"])
    co, _ = OL.lora_w_forward(c, *one("co"))
    n3 = O.addnorm_forward(n2["h"], co, p["w_mlp"], eps=eps)
    y = OL.mlp_forward(n3["x"], pm)["y"]
    n4 = O.addnorm_forward(n3["h"], y, p["w_head"], eps=eps)
    logits = n4["x"] @ head.T
    has = (tgt >= 0) / (tgt >= 0).sum()
    t = (np_(b.teacher.ids), host64(b.teacher.values))
    dkl, dlogp = layer.kl_weight * has, -layer.hard_weight * has
    fw = O.distill_forward(logits, *t, tgt, layer.scale, True)
    loss = (dkl * fw["kl"] + dlogp * fw["logp"]).sum()
    g = {}
    dl = O.distill_backward(logits, *t, dkl, tgt, dlogp, layer.scale, True)
    b4 = O.addnorm_backward(n3["h"], y, None, dl @ head, p["w_head"], eps=eps)
    bm = OL.mlp_backward(n3["x"], b4["dy"], pm)
    b3 = O.addnorm_backward(n2["h"], co, b4["dh"], bm["dX"], p["w_mlp"], eps=eps)
    parts = {"co": OL.lora_w_backward(c, b3["dy"], *one("co"))}
    br = O.attn_backward(cqn, ckn, cv, heads(parts["co"]["dX"]), csee, sc)
    dcq, g["w_cq"] = O.qkrope_backward(cq, br["dQ"], w=p["w_cq"], **nrm)
    dck, g["w_ck"] = O.qkrope_backward(ck, br["dK"], w=p["w_ck"], **nrm)
    parts["cq"] = OL.lora_w_backward(n2["x"], flat(dcq), *one("cq"))
    parts["ck"], parts["cv"] = OL.lora_w_backward(st, flat(dck), *one("ck")), OL.lora_w_backward(st, flat(br["dV"]), *one("cv"))
    b2 = O.addnorm_backward(h0, o, b3["dh"], parts["cq"]["dX"], p["w_cross"], eps=eps)
    parts["o"] = OL.lora_w_backward(a, b2["dy"], *one("o"))
    ba = O.attn_backward(q, k, v, heads(parts["o"]["dX"]), see, sc)
    dq, g["w_q"] = O.qkrope_backward(q0, ba["dQ"], w=p["w_q"], **rot)
    dk, g["w_k"] = O.qkrope_backward(k0, ba["dK"], w=p["w_k"], **rot)
    bq = OL.qkv_backward(n1["x"], flat(dq), flat(dk), flat(ba["dV"]), pq)
    g["w_attn"] = O.addnorm_backward(h0, None, b2["dh"], bq["dX"], p["w_attn"], eps=eps)["dw_in"]
    g["w_cross"], g["w_mlp"], g["w_head"] = b2["dw_in"], b3["dw_in"], b4["dw_in"]
    for n, part in parts.items():
        g["A_" + n], g["B_" + n] = part["dA"], part["dB"]
    for part, names, keys in ((bm, ("gate", "up", "down"), "gud"), (bq, ("q", "k", "v"), "qkv")):
        for n, k in zip(names, keys):
            g["A_" + n], g["B_" + n] = part["dA" + k], part["dB" + k]
    return loss, g


def _small(example):
    s = example.Sizes(T=301, S=3 * 150, docs=3, d=256, n=704, hq=4, hk=2, head=64, V=1000, K=12, r=8)
    return example.ReadingLayer(s, seed=3, b_std=0.02), example.batch(s, seed=4)


def test_against_the_chained_definitions(example):
    layer, b = _small(example)
    want, ref = _reference(layer, b)
    # the states that are not there hold anything
    for i in range(layer.s.docs):
        b.states[i * 150 + int(b.used[i]):(i + 1) * 150] = 77.0
    f = layer.forward(b)
    loss = float(layer.loss(f, b))
    got = layer.backward(f, b)
    for ws in layer.workspaces(f):
        L.lm_workspace_check(ws)
    assert abs(loss - want) <= 1e-2, (loss, want)
    assert set(got) == set(ref) == set(layer.params)
    for n in ref:
        check(n, host64(got[n]), ref[n], STEP_REL, 2 * STEP_REL)


def test_a_captured_step_beside_an_eager_one(example):
    layer, b = _small(example)

    def step():
        f = layer.forward(b)
        loss = layer.loss(f, b)
        return [loss, *layer.backward(f, b).values()]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    eager = layer.forward(b)  # (alive while the other is captured)
    layer.loss(eager, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(x, y) for x, y in zip(layer.backward(eager, b).values(), want[1:]))


def test_the_example_runs(example):
    s = example.Sizes(T=200, S=130, docs=2, d=256, n=512, hq=4, hk=1, head=128, V=500)
    losses = example.train(example.ReadingLayer(s), example.batch(s), 3, 1e-2, log=lambda line: None)
    assert len(losses) == 3 and np.isfinite(losses).all()
