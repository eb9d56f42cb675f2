"""LoRA fine-tuning of one decoder layer that reads images: packed documents of text and image tokens with three
axes of positions, normed and rotated heads, attention within each document, attention to the padded states of each
document's encoder, an MLP, a frozen output head, and a loss of two parts: the divergence from a teacher's top log
probabilities and the tokens' own log probabilities.

    python examples/reading_layer.py                       # the 8B layer's sizes, 8192 tokens, 4096 places of states
    python examples/reading_layer.py --tokens 512 --d 256 --n 704 --hq 4 --hk 2 --head-dim 64 --vocab 1000 --places 256

Weights, states and the teacher are random.  Prints the loss and the time of each step.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from bwd_lora_mlp_gb300 import layer as M  # noqa: E402
from bwd_lora_mlp_gb300 import lib as L  # noqa: E402


@dataclass
class Sizes:
    T: int       # tokens
    S: int       # places of encoder states, the same number for each document
    docs: int
    d: int
    n: int
    hq: int
    hk: int
    head: int
    V: int
    K: int = 20  # entries of the teacher
    r: int = 16


@dataclass
class Batch:
    tokens: torch.Tensor   # (T) int64
    targets: torch.Tensor  # (T) int64, negative: none
    cu: torch.Tensor       # (docs + 1) int32 offsets
    pos: torch.Tensor      # (3, T) int32: frame, row, column
    states: torch.Tensor   # (S, d) bf16
    cu_states: torch.Tensor
    used: torch.Tensor     # (docs) int32: states of each document that are there
    teacher: M.Teacher


class ReadingLayer:
    """Frozen bf16 base weights; fp32 LoRA parameters and norm weights are trained (``params``)."""

    kl_weight, hard_weight, scale = 0.7, 0.3, 0.5

    def __init__(self, s: Sizes, seed: int = 0, b_std: float = 0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.s = s
        self.embed = normal(s.V, s.d, std=1.0)
        self.head = normal(s.V, s.d, std=s.d ** -0.5)
        nq, nk = s.hq * s.head, s.hk * s.head
        self.lora, self.params = {}, {}
        for name, din, dout in (("q", s.d, nq), ("k", s.d, nk), ("v", s.d, nk), ("o", nq, s.d), ("cq", s.d, nq), ("ck", s.d, nk),
                                ("cv", s.d, nk), ("co", nq, s.d), ("gate", s.d, s.n), ("up", s.d, s.n), ("down", s.n, s.d)):
            A = normal(s.r, din, std=din ** -0.5, dtype=torch.float32)
            B = normal(dout, s.r, std=b_std, dtype=torch.float32)
            self.lora[name] = L.Lora(normal(dout, din, std=din ** -0.5), A, B, 2.0)
            self.params["A_" + name], self.params["B_" + name] = A, B
        for name in ("w_attn", "w_cross", "w_mlp", "w_head"):
            self.params[name] = torch.ones(s.d, device="cuda")
        for name in ("w_q", "w_k", "w_cq", "w_ck"):  # of a head
            self.params[name] = 1 + normal(s.head, std=0.1, dtype=torch.float32)
        pairs = s.head // 2
        i = torch.arange(pairs, device="cuda")
        self.inv_freq = (1e4 ** (-i.double() / pairs)).float()
        self.axis = (i * 3 // pairs).to(torch.int32)  # frames, rows and columns share the pairs in sections

    def rope(self, b: Batch) -> M.QkRope:
        return M.QkRope(inv_freq=self.inv_freq, pos=b.pos, axis=self.axis, norm=True, w_q=self.params["w_q"], w_k=self.params["w_k"])

    def head_norm(self, name: str) -> M.QkRope:
        return M.QkRope(norm=True, w_q=self.params[name])

    def attn(self, b: Batch) -> M.Attn:
        return M.Attn(scale=self.s.head ** -0.5, cu_docs=b.cu)

    def cross(self, b: Batch) -> M.Cross:
        return M.Cross(scale=self.s.head ** -0.5, cu_q=b.cu, cu_k=b.cu_states, k_len=b.used)

    def forward(self, b: Batch) -> dict:
        s, lo, p = self.s, self.lora, self.params
        heads = lambda t, h: t.view(-1, h, s.head)  # noqa: E731
        f = {"h0": self.embed[b.tokens]}
        f["n1"] = M.addnorm_fwd(f["h0"], None, M.AddNorm(w_in=p["w_attn"]))
        f["qkv"] = L.lora_qkv_fwd(f["n1"]["x"], lo["q"], lo["k"], lo["v"])
        f["q0"], f["k0"], f["v"] = heads(f["qkv"]["Q"], s.hq), heads(f["qkv"]["K"], s.hk), heads(f["qkv"]["V"], s.hk)
        f["rot"] = M.qkrope_fwd(f["q0"], f["k0"], self.rope(b))
        f["att"] = M.attn_fwd(f["rot"]["q"], f["rot"]["k"], f["v"], self.attn(b))
        f["a"] = f["att"]["O"].view(-1, s.hq * s.head)
        f["o"] = L.lora_o_fwd(f["a"], lo["o"])
        f["n2"] = M.addnorm_fwd(f["h0"], f["o"]["Y"], M.AddNorm(w_in=p["w_cross"]))
        f["cq"], f["ck"], f["cv"] = (L.lora_o_fwd(x, lo[n]) for x, n in ((f["n2"]["x"], "cq"), (b.states, "ck"), (b.states, "cv")))
        f["cqn"] = M.qkrope_fwd(heads(f["cq"]["Y"], s.hq), None, self.head_norm("w_cq"))["q"]
        f["ckn"] = M.qkrope_fwd(heads(f["ck"]["Y"], s.hk), None, self.head_norm("w_ck"))["q"]
        f["read"] = M.cross_fwd(f["cqn"], f["ckn"], heads(f["cv"]["Y"], s.hk), self.cross(b))
        f["c"] = f["read"]["O"].view(-1, s.hq * s.head)
        f["co"] = L.lora_o_fwd(f["c"], lo["co"])
        f["n3"] = M.addnorm_fwd(f["n2"]["h"], f["co"]["Y"], M.AddNorm(w_in=p["w_mlp"]))
        f["mlp"] = L.lora_mlp_fwd(f["n3"]["x"], lo["gate"], lo["up"], lo["down"])
        f["n4"] = M.addnorm_fwd(f["n3"]["h"], f["mlp"]["y"], M.AddNorm(w_in=p["w_head"]))
        f["logits"] = f["n4"]["x"] @ self.head.t()
        return f

    def loss(self, f: dict, b: Batch):
        """kl_weight times the mean divergence less hard_weight times the mean log probability, over the tokens with a target."""
        f["loss"] = M.distill_fwd(f["logits"], b.teacher, targets=b.targets, scale=self.scale)
        has = (b.targets >= 0).float() / (b.targets >= 0).sum().clamp(min=1)
        f["dkl"], f["dlogp"] = self.kl_weight * has, -self.hard_weight * has
        return (f["dkl"] * f["loss"]["kl"] + f["dlogp"] * f["loss"]["logp"]).sum()

    def backward(self, f: dict, b: Batch) -> dict:
        """Gradients by parameter name; the logits' buffer is overwritten by its gradient."""
        s, lo, p, g = self.s, self.lora, self.params, {}
        heads, flat = lambda t, h: t.view(-1, h, s.head), lambda t: t.view(t.shape[0], -1)  # noqa: E731
        dl = M.distill_bwd(f["logits"], b.teacher, f["loss"], f["dkl"], targets=b.targets, dlogp=f["dlogp"], scale=self.scale,
                           dlogits=f["logits"])["dlogits"]
        b4 = M.addnorm_bwd(f["n3"]["h"], f["mlp"]["y"], None, dl @ self.head, f["n4"], M.AddNorm(w_in=p["w_head"]))
        bm = L.lora_mlp_bwd(f["n3"]["x"], b4["dy"], f["mlp"], lo["gate"], lo["up"], lo["down"])
        b3 = M.addnorm_bwd(f["n2"]["h"], f["co"]["Y"], b4["dh"], bm["dX"], f["n3"], M.AddNorm(w_in=p["w_mlp"]))
        bc = L.lora_o_bwd(f["c"], b3["dy"], f["co"], lo["co"])
        br = M.cross_bwd(f["cqn"], f["ckn"], heads(f["cv"]["Y"], s.hk), heads(bc["dX"], s.hq), f["read"], self.cross(b))
        nq = M.qkrope_bwd(heads(f["cq"]["Y"], s.hq), None, br["dQ"], None, self.head_norm("w_cq"), dq_in=br["dQ"])
        nk = M.qkrope_bwd(heads(f["ck"]["Y"], s.hk), None, br["dK"], None, self.head_norm("w_ck"), dq_in=br["dK"])
        parts = {"o": None, "co": bc, "cq": L.lora_o_bwd(f["n2"]["x"], flat(nq["dq"]), f["cq"], lo["cq"]),
                 "ck": L.lora_o_bwd(b.states, flat(nk["dq"]), f["ck"], lo["ck"]),
                 "cv": L.lora_o_bwd(b.states, flat(br["dV"]), f["cv"], lo["cv"])}
        b2 = M.addnorm_bwd(f["h0"], f["o"]["Y"], b3["dh"], parts["cq"]["dX"], f["n2"], M.AddNorm(w_in=p["w_cross"]))
        parts["o"] = bo = L.lora_o_bwd(f["a"], b2["dy"], f["o"], lo["o"])
        ba = M.attn_bwd(f["rot"]["q"], f["rot"]["k"], f["v"], heads(bo["dX"], s.hq), f["att"], self.attn(b))
        bt = M.qkrope_bwd(f["q0"], f["k0"], ba["dQ"], ba["dK"], self.rope(b), dq_in=ba["dQ"], dk_in=ba["dK"])
        bq = L.lora_qkv_bwd(f["n1"]["x"], flat(bt["dq"]), flat(bt["dk"]), flat(ba["dV"]), f["qkv"], lo["q"], lo["k"], lo["v"])
        b1 = M.addnorm_bwd(f["h0"], None, b2["dh"], bq["dX"], f["n1"], M.AddNorm(w_in=p["w_attn"]))
        g["w_attn"], g["w_cross"], g["w_mlp"], g["w_head"] = b1["dw_in"], b2["dw_in"], b3["dw_in"], b4["dw_in"]
        g["w_q"], g["w_k"], g["w_cq"], g["w_ck"] = bt["dw_q"], bt["dw_k"], nq["dw_q"], nk["dw_q"]
        for name, part in parts.items():
            g["A_" + name], g["B_" + name] = part["dA"], part["dB"]
        for part, names in ((bm, ("gate", "up", "down")), (bq, ("q", "k", "v"))):
            for name in names:
                g["A_" + name], g["B_" + name] = part["dA_" + name], part["dB_" + name]
        return g

    def workspaces(self, f: dict) -> list:
        return [f[n]["ws"] for n in ("qkv", "att", "o", "cq", "ck", "cv", "read", "co", "mlp")]


def batch(s: Sizes, seed: int = 0) -> Batch:
    """Documents of about the same length, a few padding tokens behind them; each begins with an image of rows of 16 patches
    and goes on with text, which counts all three axes up together."""
    g = torch.Generator().manual_seed(seed)
    end = s.T - min(5, s.T // 10)
    cu = [end * i // s.docs for i in range(s.docs + 1)]
    pos, targets = torch.zeros(3, s.T, dtype=torch.int32), torch.full((s.T,), -1, dtype=torch.int64)
    tokens = torch.randint(s.V, (s.T,), generator=g)
    for i, (a, z) in enumerate(zip(cu, cu[1:])):
        n = (z - a) // 2
        t = torch.arange(n)
        pos[:, a:a + n] = torch.stack((torch.zeros(n, dtype=torch.int64), t // 16, t % 16))
        pos[:, a + n:z] = (n // 16 + 1 + torch.arange(z - a - n))[None]
        targets[a + n:z - 1] = tokens[a + n + 1:z]
    places = s.S // s.docs
    used = torch.randint(max(1, places // 2), places + 1, (s.docs,), generator=g, dtype=torch.int32)
    logits = torch.randn(s.T, s.V, generator=g) * 2
    lp, ids = torch.log_softmax(ReadingLayer.scale * logits, -1).topk(s.K, -1)  # (at the loss's scale)
    return Batch(tokens.cuda(), targets.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"), pos.cuda(),
                 torch.randn(s.S, s.d, generator=g).bfloat16().cuda(),
                 torch.arange(s.docs + 1, dtype=torch.int32, device="cuda") * places, used.cuda(),
                 M.Teacher(ids.to(torch.int32).cuda(), lp.cuda(), rest=True))


def train(layer: ReadingLayer, b: Batch, steps: int, lr: float, log=print) -> list:
    opt = torch.optim.Adam(list(layer.params.values()), lr=lr)
    losses = []
    for step in range(steps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        f = layer.forward(b)
        loss = layer.loss(f, b)
        for name, grad in layer.backward(f, b).items():
            layer.params[name].grad = grad
        opt.step()
        end.record()
        losses.append(float(loss))
        for ws in layer.workspaces(f):
            L.lm_workspace_check(ws)
        log("step %d  loss %.4f  %.2f ms" % (step, losses[-1], start.elapsed_time(end)))
    return losses


def main():
    ap = argparse.ArgumentParser()
    for flag, default in (("--tokens", 8192), ("--places", 4096), ("--docs", 8), ("--d", 4096), ("--n", 14336), ("--hq", 32),
                          ("--hk", 8), ("--head-dim", 128), ("--vocab", 32000), ("--entries", 20), ("--rank", 16), ("--steps", 10)):
        ap.add_argument(flag, type=int, default=default)
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args()
    s = Sizes(a.tokens, a.places, a.docs, a.d, a.n, a.hq, a.hk, a.head_dim, a.vocab, a.entries, a.rank)
    print("%d tokens in %d documents, %d places of states, %d teacher entries" % (s.T, s.docs, s.S, s.K))
    train(ReadingLayer(s), batch(s), a.steps, a.lr)


if __name__ == "__main__":
    main()
