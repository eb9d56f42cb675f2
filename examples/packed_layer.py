"""LoRA fine-tuning of one decoder layer over packed documents, every operator of the library in its
place: norm, LoRA Q/K/V, attention within each document (positions as per-head slopes), LoRA O,
residual add and norm, LoRA MLP, residual add and norm, a frozen output head, and the log
probabilities of the next tokens with their gradient written over the logits.

    python examples/packed_layer.py                        # the 8B layer's sizes, 8192 tokens
    python examples/packed_layer.py --tokens 512 --d 256 --n 704 --hq 4 --hk 2 --head-dim 64 --vocab 1000

Weights are random and the documents synthetic (each repeats a few tokens of its own), so the loss
falls from log(vocab) towards what a document's own tokens cost.  Prints the loss and the time of each
step, then the most likely continuations of the first documents.
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from bwd_lora_mlp_gb300 import layer as M  # noqa: E402
from bwd_lora_mlp_gb300 import lib as L  # noqa: E402


@dataclass
class Sizes:
    T: int
    d: int
    n: int
    hq: int
    hk: int
    head: int
    V: int
    r: int = 16


class PackedLayer:
    """Frozen bf16 base weights; fp32 LoRA parameters and norm weights are trained (``params``)."""

    def __init__(self, s: Sizes, seed: int = 0, b_std: float = 0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.s = s
        self.embed = normal(s.V, s.d, std=1.0)
        self.head = normal(s.V, s.d, std=s.d ** -0.5)
        nq, nk = s.hq * s.head, s.hk * s.head
        self.lora, self.params = {}, {}
        for name, din, dout in (("q", s.d, nq), ("k", s.d, nk), ("v", s.d, nk), ("o", nq, s.d), ("gate", s.d, s.n),
                                ("up", s.d, s.n), ("down", s.n, s.d)):
            A = normal(s.r, din, std=din ** -0.5, dtype=torch.float32)
            B = normal(dout, s.r, std=b_std, dtype=torch.float32)
            self.lora[name] = L.Lora(normal(dout, din, std=din ** -0.5), A, B, 2.0)
            self.params["A_" + name], self.params["B_" + name] = A, B
        for name in ("w_attn", "w_mlp", "w_head"):
            self.params[name] = torch.ones(s.d, device="cuda")
        # 2^-1 .. 2^-8 over the heads: scores fall with distance at a rate per head
        self.slopes = torch.exp2(-8.0 * torch.arange(1, s.hq + 1, device="cuda") / s.hq).float()

    def attn(self, cu_docs) -> M.Attn:
        return M.Attn(scale=self.s.head ** -0.5, cu_docs=cu_docs, slopes=self.slopes)

    def forward(self, tokens, cu_docs) -> dict:
        s, lo, p = self.s, self.lora, self.params
        heads = lambda t, h: t.view(-1, h, s.head)  # noqa: E731
        f = {"h0": self.embed[tokens], "cu": cu_docs}
        f["n1"] = M.addnorm_fwd(f["h0"], None, M.AddNorm(w_in=p["w_attn"]))
        f["qkv"] = L.lora_qkv_fwd(f["n1"]["x"], lo["q"], lo["k"], lo["v"])
        f["q"], f["k"], f["v"] = heads(f["qkv"]["Q"], s.hq), heads(f["qkv"]["K"], s.hk), heads(f["qkv"]["V"], s.hk)
        f["att"] = M.attn_fwd(f["q"], f["k"], f["v"], self.attn(cu_docs))
        f["a"] = f["att"]["O"].view(-1, s.hq * s.head)
        f["o"] = L.lora_o_fwd(f["a"], lo["o"])
        f["n2"] = M.addnorm_fwd(f["h0"], f["o"]["Y"], M.AddNorm(w_in=p["w_mlp"]))
        f["mlp"] = L.lora_mlp_fwd(f["n2"]["x"], lo["gate"], lo["up"], lo["down"])
        f["n3"] = M.addnorm_fwd(f["n2"]["h"], f["mlp"]["y"], M.AddNorm(w_in=p["w_head"]))
        f["logits"] = f["n3"]["x"] @ self.head.t()
        return f

    def loss(self, f: dict, targets):
        """The mean over the tokens with a target (others are negative) of -log p; and the log probabilities."""
        f["lp"] = M.logprob_fwd(f["logits"], targets)
        count = (targets >= 0).sum().clamp(min=1)
        f["dlogp"] = torch.full_like(f["lp"]["logp"], -1.0) / count
        return -f["lp"]["logp"].sum() / count

    def backward(self, f: dict, targets) -> dict:
        """Gradients by parameter name; the logits' buffer is overwritten by its gradient."""
        s, lo, p, g = self.s, self.lora, self.params, {}
        dl = M.logprob_bwd(f["logits"], targets, f["lp"], f["dlogp"], dlogits=f["logits"])["dlogits"]
        b3 = M.addnorm_bwd(f["n2"]["h"], f["mlp"]["y"], None, dl @ self.head, f["n3"], M.AddNorm(w_in=p["w_head"]))
        bm = L.lora_mlp_bwd(f["n2"]["x"], b3["dy"], f["mlp"], lo["gate"], lo["up"], lo["down"])
        b2 = M.addnorm_bwd(f["h0"], f["o"]["Y"], b3["dh"], bm["dX"], f["n2"], M.AddNorm(w_in=p["w_mlp"]))
        bo = L.lora_o_bwd(f["a"], b2["dy"], f["o"], lo["o"])
        ba = M.attn_bwd(f["q"], f["k"], f["v"], bo["dX"].view(-1, s.hq, s.head), f["att"], self.attn(f["cu"]))
        bq = L.lora_qkv_bwd(f["n1"]["x"], ba["dQ"].view(-1, s.hq * s.head), ba["dK"].view(-1, s.hk * s.head),
                            ba["dV"].view(-1, s.hk * s.head), f["qkv"], lo["q"], lo["k"], lo["v"])
        b1 = M.addnorm_bwd(f["h0"], None, b2["dh"], bq["dX"], f["n1"], M.AddNorm(w_in=p["w_attn"]))
        g["w_attn"], g["w_mlp"], g["w_head"] = b1["dw_in"], b2["dw_in"], b3["dw_in"]
        g["A_o"], g["B_o"] = bo["dA"], bo["dB"]
        for part, names in ((bm, ("gate", "up", "down")), (bq, ("q", "k", "v"))):
            for name in names:
                g["A_" + name], g["B_" + name] = part["dA_" + name], part["dB_" + name]
        return g


def packed_documents(T: int, V: int, seed: int = 0):
    """Documents of 40 to 1000 tokens, each from 8 tokens of its own, packed into T; the rest is padding.
    Returns tokens, next-token targets (-1: none) and the offsets."""
    g = torch.Generator().manual_seed(seed)
    tokens, targets, cu = torch.zeros(T, dtype=torch.int64), torch.full((T,), -1, dtype=torch.int64), [0]
    while True:
        n = int(torch.randint(40, 1001, (1,), generator=g))
        if cu[-1] + n > T:
            n = T - cu[-1]
            if n < 40:
                break
        own = torch.randint(V, (8,), generator=g)
        doc = own[torch.randint(8, (n,), generator=g)]
        tokens[cu[-1]:cu[-1] + n] = doc
        targets[cu[-1]:cu[-1] + n - 1] = doc[1:]
        cu.append(cu[-1] + n)
    return tokens.cuda(), targets.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda")


def train(layer: PackedLayer, tokens, targets, cu_docs, steps: int, lr: float, log=print) -> list:
    opt = torch.optim.Adam(list(layer.params.values()), lr=lr)
    losses = []
    for step in range(steps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f = layer.forward(tokens, cu_docs)
        loss = layer.loss(f, targets)
        for name, grad in layer.backward(f, targets).items():
            layer.params[name].grad = grad
        opt.step()
        b.record()
        losses.append(float(loss))
        for ws in (f["qkv"]["ws"], f["att"]["ws"], f["o"]["ws"], f["mlp"]["ws"]):
            L.lm_workspace_check(ws)
        log("step %d  loss %.4f  %.2f ms" % (step, losses[-1], a.elapsed_time(b)))
    return losses


def continuations(layer: PackedLayer, tokens, cu_docs, docs: int, k: int = 5) -> dict:
    """The k most likely next tokens after the last token of each of the first documents."""
    f = layer.forward(tokens, cu_docs)
    last = (cu_docs[1:docs + 1] - 1).long()
    return M.logprob_fwd(f["logits"][last], torch.full_like(last, -1), k=k)


def main():
    ap = argparse.ArgumentParser()
    for flag, default in (("--tokens", 8192), ("--d", 4096), ("--n", 14336), ("--hq", 32), ("--hk", 8), ("--head-dim", 128),
                          ("--vocab", 32000), ("--rank", 16), ("--steps", 10)):
        ap.add_argument(flag, type=int, default=default)
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args()
    s = Sizes(a.tokens, a.d, a.n, a.hq, a.hk, a.head_dim, a.vocab, a.rank)
    tokens, targets, cu = packed_documents(s.T, s.V)
    layer = PackedLayer(s)
    print("%d tokens, %d documents, log(vocab) = %.3f" % (s.T, cu.numel() - 1, math.log(s.V)))
    train(layer, tokens, targets, cu, a.steps, a.lr)
    docs = min(3, cu.numel() - 1)
    top = continuations(layer, tokens, cu, docs)
    for i in range(docs):
        print("document %d: next of %s with log p %s" % (i, top["top_ids"][i].tolist(),
                                                         [round(x, 3) for x in top["top_logp"][i].tolist()]))


if __name__ == "__main__":
    main()
