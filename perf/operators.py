"""Cases of the operators around the LoRA projections of a decoder layer, in their plain form and
through the framework's entry points: attention over packed documents with capped or
distance-biased scores (attn), residual add with the norms before and after a block (addnorm),
and log probabilities, entropy and top alternatives of given tokens (logprob).

A case with "train" runs forward and backward as one training step does; the others run the
forward alone.  The plain forms compute in fp32 with elementary torch operations and round once.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------------
# cases


def _attn(name, T, hq, hk, D, train=True, docs=0, pad=0, prefix=False, causal=True, window=0, cap=0.0, bias=False,
          fused=False, layout=1):
    return {"name": name, "op": "attn", "T": T, "hq": hq, "hk": hk, "D": D, "train": train, "docs": docs, "pad": pad,
            "prefix": prefix, "causal": causal, "window": window, "cap": cap, "bias": bias, "fused": fused,
            "layout": layout}


def _addnorm(name, T, d, train=True, add=True, post=True, gate=False, f32=False, offset=0.0, alpha=1.0):
    return {"name": name, "op": "addnorm", "T": T, "d": d, "train": train, "add": add, "post": post, "gate": gate,
            "f32": f32, "offset": offset, "alpha": alpha}


def _logprob(name, T, V, train=True, k=0, f32=False, scale=1.0, pad=0):
    return {"name": name, "op": "logprob", "T": T, "V": V, "train": train, "k": k, "f32": f32, "scale": scale,
            "pad": pad}


def listed():
    return [
        # one short prompt scored by the 32/8-head layer: latency
        _attn("attn fwd 128", 128, 32, 8, 128, train=False),
        # evaluation of one full-length sequence with capped scores
        _attn("attn fwd 4096 cap", 4096, 32, 8, 128, train=False, cap=30.0),
        # the framework's training step: 8192 tokens in one causal sequence, 32/8 heads of 128
        _attn("attn train 8192", 8192, 32, 8, 128),
        # the same tokens as packed documents with a padded tail, read from the fused QKV buffer
        _attn("attn train 8192 docs", 8192, 32, 8, 128, docs=14, pad=83, fused=True, layout=3),
        # distance-biased scores in a sliding window, small heads, an odd length
        _attn("attn train 2999 bias", 2999, 16, 16, 64, window=1024, bias=True),
        # instruction tuning with bidirectional prompts: packed prefix masks, capped scores, heads of 80
        _attn("attn train 4097 prefix", 4097, 20, 4, 80, docs=9, prefix=True, cap=20.0, layout=5),
        # the norm step of a few new tokens: latency
        _addnorm("addnorm fwd 16x4096", 16, 4096, train=False),
        # the framework's training step: norms before and after the block, per-channel gate
        _addnorm("addnorm train 8192x4096", 8192, 4096, gate=True, alpha=0.5),
        # an odd token count, an fp32 residual stream, no norm after the block
        _addnorm("addnorm train 3001x8192", 3001, 8192, post=False, f32=True, offset=1.0),
        # sampling: alternatives of four rows of fp32 logits, latency
        _logprob("logprob fwd 4x131072", 4, 131072, train=False, k=20, f32=True, scale=1.25),
        # fine-tuning loss over an odd vocabulary whose rows are not aligned
        _logprob("logprob train 1000x50257", 1000, 50257, k=5),
        # policy-gradient loss with entropy over a large vocabulary
        _logprob("logprob train 4096x131072", 4096, 131072, k=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "addnorm", "logprob"])
    train = rng.random() < 0.7
    if op == "attn":
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        # (a query that sees one key has a gradient of exactly nothing, and rounding noise has no relative error:
        # training draws start where most queries see many keys)
        T = _log_int(rng, 64 if train else 1, min(8192, int(8192 * math.sqrt(32 / hq))))
        docs = rng.choice([0, 0, 1 + T // 2000, 1 + T // 300, 1 + T // 60])
        causal = rng.random() < 0.85
        return {"op": "attn", "T": T, "hq": hq, "hk": hk, "D": D, "train": train, "docs": docs,
                "pad": rng.randint(0, T // 8) if docs else 0, "prefix": bool(docs and causal and rng.random() < 0.4),
                "causal": causal, "window": rng.choice([0, 0, 0, _log_int(rng, 32, 2048)]),
                "cap": rng.choice([0.0, 0.0, 20.0, 50.0]), "bias": rng.random() < 0.3, "fused": rng.random() < 0.4,
                "layout": rng.randint(1, 1 << 20)}
    if op == "addnorm":
        d = 32 * _log_int(rng, 8, 384)
        T = _log_int(rng, 1, min(16384, (8192 * 4096) // d))
        add = rng.random() < 0.85
        return {"op": "addnorm", "T": T, "d": d, "train": train, "add": add, "post": add and rng.random() < 0.6,
                "gate": add and rng.random() < 0.4, "f32": rng.random() < 0.3, "offset": rng.choice([0.0, 0.0, 1.0]),
                "alpha": rng.choice([1.0, 0.5, 0.22])}
    V = _log_int(rng, 300, 160000)
    f32 = rng.random() < 0.3
    T = _log_int(rng, 1, max(1, min(8192, (1 << 28) // V)))
    return {"op": "logprob", "T": T, "V": V, "train": train, "k": rng.choice([0, 0, 1, 5, 20, 32]), "f32": f32,
            "scale": rng.choice([1.0, 1.0, 0.7, 1.4]), "pad": rng.choice([0, 0, 0, 7, 64])}


def _cuts(case):
    """Document boundaries (docs + 1 offsets; the padded tail belongs to none) and prefix lengths."""
    rng = random.Random(case["layout"])
    end = case["T"] - case["pad"]
    inner = sorted(rng.randint(0, end) for _ in range(case["docs"] - 1))
    cu = [0] + inner + [end]
    return cu, [rng.randint(0, (b - a) // 2) for a, b in zip(cu, cu[1:])]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    T, W = case["T"], case["window"]
    cu, pre = _cuts(case) if case["docs"] else ([0, T], [0])
    n = 0
    for s, e, p in zip(cu, cu[1:], pre if case["prefix"] else [0] * len(cu)):
        for i in range(s, e):
            hi = max(i + 1, s + p) if case["causal"] else e
            n += (min(hi, i + W) - max(s, i - W + 1)) if W else hi - s
    return n


def work(case):
    T = case["T"]
    if case["op"] == "attn":
        hq, hk, D, pairs = case["hq"], case["hk"], case["D"], _pairs(case)
        fwd = T * (2 * hq + 2 * hk) * D * 2 + T * hq * 4
        bwd = T * (2 * hq + 2 * hk) * D * 2
        return {"bytes": fwd + (bwd if case["train"] else 0), "flops": (14 if case["train"] else 4) * D * hq * pairs}
    if case["op"] == "addnorm":
        d, hb = case["d"], 4 if case["f32"] else 2
        fwd = hb + 2 + (hb + 2 if case["add"] else 0)          # h, x; y and the sum
        bwd = 2 * hb + 2 + (2 if case["add"] else 0)           # the stream's gradient in and out, dx; dy
        return {"bytes": T * d * (fwd + (bwd if case["train"] else 0)), "flops": T * d * (40 if case["train"] else 12)}
    es = 4 if case["f32"] else 2
    return {"bytes": T * case["V"] * es * (2 if case["train"] else 1) + T * (24 + 8 * case["k"]),
            "flops": T * case["V"] * (14 if case["train"] else 7)}


# ---------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    T = case["T"]
    s = {"case": case}
    if case["op"] == "attn":
        hq, hk, D = case["hq"], case["hk"], case["D"]
        # with a cap the scores reach its bend; without one they have the spread of trained heads
        std = 3.0 if case["cap"] else 2.0
        if case["fused"]:
            qkv = normal(T, hq + 2 * hk, D)
            qkv[:, :hq] *= std
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            s["q"], s["k"], s["v"] = normal(T, hq, D, std=std), normal(T, hk, D), normal(T, hk, D)
        s["dO"] = normal(T, hq, D, std=0.01) if case["train"] else None
        s["cu"] = s["prefix"] = s["slopes"] = None
        if case["docs"]:
            cu, pre = _cuts(case)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            if case["prefix"]:
                s["prefix"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
        if case["bias"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device="cuda")
    elif case["op"] == "addnorm":
        d = case["d"]
        hd = torch.float32 if case["f32"] else torch.bfloat16
        s["h"] = normal(T, d, std=2.0, dtype=hd)
        s["y"] = normal(T, d, std=0.5) if case["add"] else None
        s["w_in"] = (1 - case["offset"] + normal(d, std=0.1)).to(torch.bfloat16)
        s["w_post"] = (1 - case["offset"] + normal(d, std=0.1)).to(torch.bfloat16) if case["post"] else None
        s["gate"] = normal(d, std=0.5) if case["gate"] else None
        if case["train"]:
            s["dh"], s["dx"] = normal(T, d, std=0.01, dtype=hd), normal(T, d, std=0.01)
    else:
        V = case["V"]
        full = normal(T, V + case["pad"], std=3.0, dtype=torch.float32 if case["f32"] else torch.bfloat16)
        s["logits"] = full[:, :V]
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        t[torch.rand(T, generator=g, device="cuda") < 0.1] = -100
        s["targets"] = t
        if case["train"]:
            s["dlogp"] = torch.randn(T, generator=g, device="cuda") / T
            s["dent"] = torch.randn(T, generator=g, device="cuda") * (0.1 / T)
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _attn_own, "addnorm": _addnorm_own, "logprob": _logprob_own}[op](state)
    return {"attn": _attn_plain, "addnorm": _addnorm_plain, "logprob": _logprob_plain}[op](state)


def _attn_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    a = M.Attn(scale=c["D"] ** -0.5, cap=c["cap"], causal=c["causal"], window=c["window"], cu_docs=s["cu"],
               prefix=s["prefix"], slopes=s["slopes"])
    fw = M.attn_fwd(s["q"], s["k"], s["v"], a, train=c["train"], ws=s.get("ws"))
    s["ws"] = fw["ws"]
    out = {"O": fw["O"], "lse": fw["lse"]}
    if c["train"]:
        out.update(M.attn_bwd(s["q"], s["k"], s["v"], s["dO"], fw, a))
    return out


def _visible(c, cu, prefix):
    """(T, T) truth values: query i (row) sees key j (column)."""
    i = torch.arange(c["T"], device="cuda")
    far = i[:, None] - i[None, :]
    see = (far >= 0) if c["causal"] else torch.ones_like(far, dtype=torch.bool)
    if cu is not None:
        doc = (i[:, None] >= cu[None, :]).sum(1) - 1
        if prefix is not None:
            at = doc.clamp(0, prefix.numel() - 1)
            see = see | (i < cu[at] + prefix[at])[None, :]
        inside = doc < cu.numel() - 1
        see = see & (doc[:, None] == doc[None, :]) & inside[None, :]
    if c["window"]:
        see = see & (far.abs() < c["window"])
    return see


def _attn_plain(s):
    c = s["case"]
    T, hq, hk, D, cap = c["T"], c["hq"], c["hk"], c["D"], c["cap"]
    scale = D ** -0.5

    def heads(x):  # (T, h, D) -> (hk, h / hk, T, D) fp32
        return x.float().view(T, hk, -1, D).permute(1, 2, 0, 3)

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    S = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    bend = None
    if cap:
        S = S.div_(cap).tanh_()
        bend = 1 - S * S if c["train"] else None
        S = S.mul_(cap)
    if s["slopes"] is not None:
        i = torch.arange(T, device="cuda", dtype=torch.float32)
        S = S - s["slopes"].view(hk, -1, 1, 1) * (i[:, None] - i[None, :]).abs()
    S = S.masked_fill_(~_visible(c, s["cu"], s["prefix"]), -math.inf)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = P.sum(-1, keepdim=True)
    P = P.div_(torch.where(l == 0, torch.ones_like(l), l))
    lse = (m + l.log()).view(hq, T)

    def tokens(x):  # (hk, n, T, D) -> (T, hk n, D) bf16
        return x.permute(2, 0, 1, 3).reshape(T, -1, D).to(torch.bfloat16)

    O = torch.matmul(P, v)
    out = {"O": tokens(O), "lse": lse}
    if c["train"]:
        dO = heads(s["dO"])
        dV = torch.matmul(P.transpose(-1, -2), dO).sum(1, keepdim=True)
        dS = torch.matmul(dO, v.transpose(-1, -2)).sub_((dO * O).sum(-1, keepdim=True)).mul_(P)
        del P
        if bend is not None:
            dS = dS.mul_(bend)
        dS = dS.mul_(scale)
        out["dQ"] = tokens(torch.matmul(dS, k))
        out["dK"] = tokens(torch.matmul(dS.transpose(-1, -2), q).sum(1, keepdim=True))
        out["dV"] = tokens(dV)
    return out


def _addnorm_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    n = M.AddNorm(w_in=s["w_in"], w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"], eps=1e-5, w_offset=c["offset"])
    fw = M.addnorm_fwd(s["h"], s["y"], n)
    out = {"h": fw["h"], "x": fw["x"]}
    if c["train"]:
        bw = M.addnorm_bwd(s["h"], s["y"], s["dh"], s["dx"], fw, n, ws=s.get("ws"))
        s["ws"] = bw.pop("ws")
        out["grads"] = {k: t for k, t in bw.items() if t is not None}
    return out


def _addnorm_plain(s):
    c = s["case"]
    d, alpha, off, eps = c["d"], c["alpha"], c["offset"], 1e-5
    h = s["h"].float()
    w_in = s["w_in"].float() + off
    y = w_post = gate = None
    if c["add"]:
        y = s["y"].float()
        n = y
        if c["post"]:
            w_post = s["w_post"].float() + off
            ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
            n = y * ry * w_post
        if c["gate"]:
            gate = s["gate"].float()
        h = h + alpha * (n if gate is None else gate * n)
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + eps)
    hd, bf = s["h"].dtype, torch.bfloat16
    out = {"h": h.to(hd), "x": (h * r * w_in).to(bf)}
    if c["train"]:
        dx = s["dx"].float()
        t = dx * w_in
        g = s["dh"].float() + r * (t - h * (r * r) * (t * h).mean(-1, keepdim=True))
        grads = {"dh": g.to(hd), "dw_in": (dx * (h * r)).sum(0)}
        if c["add"]:
            dn = alpha * (g if gate is None else g * gate)
            if gate is not None:
                grads["dgate"] = (alpha * g * n).sum(0)
            if c["post"]:
                grads["dw_post"] = (dn * (y * ry)).sum(0)
                t = dn * w_post
                dn = ry * (t - y * (ry * ry) * (t * y).mean(-1, keepdim=True))
            grads["dy"] = dn.to(bf)
        out["grads"] = grads
    return out


def _logprob_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    fw = M.logprob_fwd(s["logits"], s["targets"], k=c["k"], scale=c["scale"])
    out = {n: fw[n] for n in ("logp", "entropy", "lse") + (("top_ids", "top_logp") if c["k"] else ())}
    if c["train"]:
        out["dlogits"] = M.logprob_bwd(s["logits"], s["targets"], fw, s["dlogp"], s["dent"], scale=c["scale"])["dlogits"]
    return out


def _logprob_plain(s):
    c = s["case"]
    x = s["logits"].float() * c["scale"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    z = e.sum(-1, keepdim=True)
    lse = m + z.log()
    p = e / z
    ent = z.log().squeeze(-1) - (p * (x - m)).sum(-1)
    t = s["targets"]
    has = (t >= 0) & (t < c["V"])
    at = torch.where(has, t, torch.zeros_like(t))[:, None]
    logp = torch.where(has, (x.gather(1, at) - lse).squeeze(1), torch.zeros_like(ent))
    out = {"logp": logp, "entropy": ent, "lse": lse.squeeze(1)}
    if c["k"]:
        order = torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices[:, :c["k"]]
        out["top_ids"] = order.to(torch.int32)
        out["top_logp"] = x.gather(1, order) - lse
    if c["train"]:
        g = torch.where(has, s["dlogp"], torch.zeros_like(ent))[:, None]
        dx = -p * (g + s["dent"][:, None] * (x - lse + ent[:, None]))
        dx.scatter_add_(1, at, g)
        out["dlogits"] = (dx * c["scale"]).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, gradients by differentiation of the forward


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _attn_exact, "addnorm": _addnorm_exact, "logprob": _logprob_exact}[case["op"]](case, s)


def _attn_exact(c, s):
    T, hq, hk, D = c["T"], c["hq"], c["hk"], c["D"]
    cu, pre = _cuts(c) if c["docs"] else ([0, T], [0])
    lo, hi = [0] * T, [0] * T  # each query's interval of keys
    for d, (a, b) in enumerate(zip(cu, cu[1:])):
        for i in range(a, b):
            lo[i] = max(a, i - c["window"] + 1) if c["window"] else a
            hi[i] = max(i + 1, a + pre[d] if c["prefix"] else 0) if c["causal"] else b
            hi[i] = min(hi[i], i + c["window"]) if c["window"] else hi[i]
    j = torch.arange(T, device="cuda")
    lo, hi = (torch.tensor(x, device="cuda")[:, None] for x in (lo, hi))
    hidden = (j < lo) | (j >= hi)
    empty = (lo >= hi).squeeze(1)
    O = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device="cuda")
    grads = {n: torch.zeros(T, h, D, dtype=torch.float64, device="cuda") for n, h in (("dQ", hq), ("dK", hk), ("dV", hk))}
    for h in range(hq):
        q, k, v = (s[n][:, at].double().requires_grad_(c["train"]) for n, at in (("q", h), ("k", h * hk // hq), ("v", h * hk // hq)))
        z = q @ k.T / math.sqrt(D)
        if c["cap"]:
            z = c["cap"] * torch.tanh(z / c["cap"])
        if c["bias"]:
            z = z - s["slopes"][h].double() * (j[:, None] - j[None, :]).abs()
        z = z.masked_fill(hidden, -math.inf)
        z = torch.where(empty[:, None], torch.zeros_like(z), z)
        o = torch.where(empty[:, None], torch.zeros_like(q), torch.softmax(z, -1) @ v)
        O[:, h] = o.detach()
        lse[h] = torch.where(empty, lse[h], torch.logsumexp(z.detach(), -1))
        if c["train"]:
            dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dO"][:, h].double())
            grads["dQ"][:, h] += dq
            grads["dK"][:, h * hk // hq] += dk
            grads["dV"][:, h * hk // hq] += dv
        del z, o
    return {"O": O, "lse": lse, **(grads if c["train"] else {})}


def _addnorm_exact(c, s):
    leaf = {n: s[n].double().requires_grad_(c["train"]) for n in ("h", "y", "w_in", "w_post", "gate") if s[n] is not None}

    def norm(a, w):
        return a / torch.sqrt(torch.mean(a ** 2, -1, keepdim=True) + 1e-5) * (w + c["offset"])

    h = leaf["h"]
    if c["add"]:
        b = norm(leaf["y"], leaf["w_post"]) if c["post"] else leaf["y"]
        h = h + c["alpha"] * b * leaf.get("gate", 1.0)
    x = norm(h, leaf["w_in"])
    out = {"h": h.detach(), "x": x.detach()}
    if c["train"]:
        names = list(leaf)
        got = torch.autograd.grad((h, x), [leaf[n] for n in names], (s["dh"].double(), s["dx"].double()))
        out["grads"] = {"d" + n: t for n, t in zip(names, got)}
    return out


def _logprob_exact(c, s):
    if c["T"] * c["V"] > 1 << 30:
        return None
    x = s["logits"].double().requires_grad_(c["train"])
    ls = torch.log_softmax(x * c["scale"], -1)
    ent = -(ls.exp() * ls).sum(-1)
    t = s["targets"]
    logp = torch.where(t < 0, torch.zeros_like(ent), ls.gather(1, t.clamp(min=0)[:, None]).squeeze(1))
    out = {"logp": logp.detach(), "entropy": ent.detach(), "lse": torch.logsumexp(x.detach() * c["scale"], -1)}
    if c["k"]:
        out["top_ids"] = None
        out["top_logp"] = torch.topk(ls.detach(), c["k"], -1).values
    if c["train"]:
        out["dlogits"], = torch.autograd.grad((logp, ent), x, (s["dlogp"].double(), s["dent"].double()))
    return out
