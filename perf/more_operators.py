"""Cases of three more operators of a LoRA training step, in their plain form and through the framework's
entry points: norms of query and key heads with the rotation by position in the same pass (qkrope),
attention to the states of an encoder of another length (cross), and distillation from a teacher's top
logits with the loss of given tokens beside it (distill).

A case with "train" runs forward and backward as one training step does; the others run the
forward alone.  The plain forms compute in fp32 with elementary torch operations (angles in 64 bits) and
round once.
"""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------------------------
# cases


def _qkrope(name, T, hq, hk, d, train=True, rot=None, axes=1, inter=False, norm=True, w32=False, offset=0.0, far=0,
            fused=False, wide=False):
    return {"name": name, "op": "qkrope", "T": T, "hq": hq, "hk": hk, "d": d, "train": train, "rot": d if rot is None else rot,
            "axes": axes, "inter": inter, "norm": norm, "w32": w32, "offset": offset, "far": far, "fused": fused,
            "wide": wide}


def _cross(name, Tq, Tk, hq, hk, d, train=True, docs=0, padded=False, cap=0.0, fused=False, layout=1):
    return {"name": name, "op": "cross", "Tq": Tq, "Tk": Tk, "hq": hq, "hk": hk, "d": d, "train": train, "docs": docs,
            "padded": padded, "cap": cap, "fused": fused, "layout": layout}


def _distill(name, T, V, K, train=True, f32=False, scale=1.0, rest=False, hard=False, pad=0):
    return {"name": name, "op": "distill", "T": T, "V": V, "K": K, "train": train, "f32": f32, "scale": scale,
            "rest": rest, "hard": hard, "pad": pad}


def listed():
    return [
        # a few new tokens of the 32/8-head layer: latency
        _qkrope("qkrope fwd 16", 16, 32, 8, 128, train=False),
        # the framework's training step: normed and rotated heads, read from the fused QKV buffer
        _qkrope("qkrope train 8192", 8192, 32, 8, 128, fused=True),
        # tokens of images among text: three axes of positions, heads of 80, an odd count, no norm
        _qkrope("qkrope train 4097 axes", 4097, 20, 4, 80, axes=3, norm=False),
        # long context: far positions, the first half of each head rotated in neighbouring pairs, fp32 weights
        _qkrope("qkrope train 16384 far", 16384, 32, 8, 128, rot=64, inter=True, w32=True, far=1 << 20, wide=True),
        # one generated token of a layer that looks at an encoder's 8192 states: latency
        _cross("cross fwd 1x8192", 1, 8192, 32, 8, 128, train=False),
        # 64 sequences generating at once, each with its own padded 1024 encoder states
        _cross("cross fwd 64x65536", 64, 65536, 32, 8, 128, train=False, docs=64, padded=True),
        # a training sequence that looks at a long encoder's states
        _cross("cross train 8192x4096", 8192, 4096, 32, 8, 128, fused=True),
        # packed documents, each with its own padded states; heads of 80, capped scores, odd sizes
        _cross("cross train 4097x4113 docs", 4097, 9 * 457, 20, 4, 80, docs=9, padded=True, cap=20.0, layout=5),
        # four rows of fp32 logits against a teacher's 20: latency
        _distill("distill fwd 4x131072", 4, 131072, 20, train=False, f32=True, scale=1.25),
        # the example's vocabulary at a temperature, with the tokens' own loss beside it
        _distill("distill train 8192x32000", 8192, 32000, 32, scale=0.5, hard=True),
        # an odd vocabulary whose rows are not aligned; what the teacher leaves is one more outcome
        _distill("distill train 1000x50257", 1000, 50257, 20, rest=True),
        # a large vocabulary, 64 teacher entries, what they leave, and the tokens' own loss
        _distill("distill train 4096x131072", 4096, 131072, 64, rest=True, hard=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qkrope", "cross", "cross", "distill"])
    train = rng.random() < 0.7
    if op == "qkrope":
        d = rng.choice([32, 64, 72, 80, 96, 128, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        T = _log_int(rng, 1, min(32768, (16384 * 40 * 128) // ((hq + hk) * d)))
        axes = rng.choice([1, 1, 2, 3])
        return {"op": "qkrope", "T": T, "hq": hq, "hk": hk, "d": d, "train": train,
                "rot": rng.choice([d, d, d, d // 16 * 8]), "axes": axes, "inter": rng.random() < 0.3,
                "norm": rng.random() < 0.7, "w32": rng.random() < 0.3, "offset": rng.choice([0.0, 0.0, 1.0]),
                "far": rng.choice([0, 0, 1000, 1 << 17, 1 << 24]), "fused": rng.random() < 0.5, "wide": rng.random() < 0.5}
    if op == "cross":
        d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 5])
        most = (1 << 30) // hq
        Tk = _log_int(rng, 64, 32768)
        Tq = _log_int(rng, 64 if train else 1, max(65, min(16384, most // Tk)))
        docs = rng.choice([0, 0, 1 + min(Tq, Tk) // 2000, 1 + min(Tq, Tk) // 100])
        if docs:  # (each document's states have a place of the same size, or are packed)
            Tk = (Tk + docs - 1) // docs * docs
        return {"op": "cross", "Tq": Tq, "Tk": Tk, "hq": hq, "hk": hk, "d": d, "train": train, "docs": docs,
                "padded": bool(docs) and rng.random() < 0.5, "cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
                "fused": rng.random() < 0.4, "layout": rng.randint(1, 1 << 20)}
    V = _log_int(rng, 300, 160000)
    T = _log_int(rng, 1, max(1, min(8192, (1 << 28) // V)))
    return {"op": "distill", "T": T, "V": V, "K": rng.choice([1, 5, 20, 32, 64, 100, 128]), "train": train,
            "f32": rng.random() < 0.3, "scale": rng.choice([1.0, 1.0, 0.5, 1.4]), "rest": rng.random() < 0.5,
            "hard": rng.random() < 0.5, "pad": rng.choice([0, 0, 0, 7, 64])}


def _segments(case):
    """Query offsets (docs + 1), key offsets and each document's key count."""
    rng = random.Random(case["layout"])
    n = case["docs"]
    if not n:
        return [0, case["Tq"]], [0, case["Tk"]], [case["Tk"]]

    def cuts(total):  # no part smaller than half of an even one
        even = total / n
        return [0] + [int(round(even * (i + rng.uniform(-0.25, 0.25)))) for i in range(1, n)] + [total]

    cu_q = list(range(n + 1)) if case["Tq"] == n else cuts(case["Tq"])
    if case["padded"]:
        size = case["Tk"] // n
        return cu_q, [i * size for i in range(n + 1)], [rng.randint(max(1, size // 2), size) for _ in range(n)]
    cu_k = cuts(case["Tk"])
    return cu_q, cu_k, [b - a for a, b in zip(cu_k, cu_k[1:])]


def work(case):
    if case["op"] == "qkrope":
        n = case["T"] * (case["hq"] + case["hk"]) * case["d"]
        pos = case["T"] * case["axes"] * (8 if case["wide"] else 4)
        steps = (2 + (3 if case["norm"] else 2)) if case["train"] else 2  # forward; x (with a norm), dy and dx
        return {"bytes": n * 2 * steps + pos * (2 if case["train"] else 1),
                "flops": n * ((9 if case["norm"] else 3) + (20 if case["norm"] else 3) * case["train"])}
    if case["op"] == "cross":
        hq, hk, d = case["hq"], case["hk"], case["d"]
        cu_q, _, lens = _segments(case)
        pairs = sum((b - a) * n for a, b, n in zip(cu_q, cu_q[1:], lens))
        q, k = case["Tq"] * hq * d * 2, sum(lens) * hk * d * 2
        fwd, bwd = 2 * q + 2 * k + case["Tq"] * hq * 4, 2 * q + 2 * k
        return {"bytes": fwd + (bwd if case["train"] else 0), "flops": (14 if case["train"] else 4) * d * hq * pairs}
    n, es = case["T"] * case["V"], 4 if case["f32"] else 2
    return {"bytes": n * es * (2 if case["train"] else 1) + case["T"] * (case["K"] * 8 + 24),
            "flops": n * (9 if case["train"] else 4)}


# ---------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    return {"qkrope": _qkrope_inputs, "cross": _cross_inputs, "distill": _distill_inputs}[case["op"]](case, g, normal)


def _qkrope_inputs(c, g, normal):
    T, hq, hk, d, r = c["T"], c["hq"], c["hk"], c["d"], c["rot"] // 2
    s = {"case": c}
    if c["fused"]:
        qkv = normal(T, hq + 2 * hk, d, std=2.0)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
    else:
        s["q"], s["k"] = normal(T, hq, d, std=2.0), normal(T, hk, d, std=2.0)
    i = torch.arange(r, device="cuda")
    s["inv_freq"] = (1e6 ** (-i.double() / r)).float()
    t = torch.arange(T, device="cuda")
    if c["axes"] == 1:  # packed documents, each counted from its start
        pos, s["axis"] = t % 5000, None
    else:  # images of 24 x 32 patches: frames, rows, columns; the axes share the pairs in sections
        grid = [t // 768, t // 32 % 24, t % 32]
        pos = torch.stack(grid[-c["axes"]:])
        s["axis"] = (i * c["axes"] // r).to(torch.int32)
    s["pos"] = (pos + c["far"]).to(torch.int64 if c["wide"] else torch.int32)
    wt = torch.float32 if c["w32"] else torch.bfloat16
    s["w_q"] = (1 - c["offset"] + normal(d, std=0.1, dtype=wt)).to(wt) if c["norm"] else None
    s["w_k"] = (1 - c["offset"] + normal(d, std=0.1, dtype=wt)).to(wt) if c["norm"] else None
    if c["train"]:
        s["dq"], s["dk"] = normal(T, hq, d, std=0.01), normal(T, hk, d, std=0.01)
    return s


def _cross_inputs(c, g, normal):
    Tq, Tk, hq, hk, d = c["Tq"], c["Tk"], c["hq"], c["hk"], c["d"]
    s = {"case": c}
    # with a cap the scores reach its bend; without one they have the spread of trained heads
    s["q"] = normal(Tq, hq, d, std=3.0 if c["cap"] else 2.0)
    if c["fused"]:  # keys and values of the encoder's states in one buffer
        kv = normal(Tk, 2 * hk, d)
        s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
    else:
        s["k"], s["v"] = normal(Tk, hk, d), normal(Tk, hk, d)
    s["dO"] = normal(Tq, hq, d, std=0.01) if c["train"] else None
    s["cu_q"] = s["cu_k"] = s["k_len"] = None
    if c["docs"]:
        cu_q, cu_k, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in _segments(c))
        s["cu_q"], s["cu_k"], s["k_len"] = cu_q, cu_k, lens if c["padded"] else None
    return s


def _distill_inputs(c, g, normal):
    T, V, K = c["T"], c["V"], c["K"]
    s = {"case": c}
    full = normal(T, V + c["pad"], std=2.5, dtype=torch.float32 if c["f32"] else torch.bfloat16)
    s["logits"] = full[:, :V]
    # a teacher that the student resembles: its K largest logits, or their log probabilities
    z = s["logits"].float() + torch.randn(T, V, generator=g, device="cuda")
    top, ids = z.topk(min(K, V), -1)
    s["teacher"] = (top - z.logsumexp(-1, keepdim=True)) if c["rest"] else top
    none = torch.rand(T, 1, generator=g, device="cuda") < 0.05  # rows without a teacher
    short = torch.rand(T, 1, generator=g, device="cuda") < 0.2   # and rows with half of the entries
    at = torch.arange(ids.shape[1], device="cuda")[None]
    s["ids"] = ids.masked_fill(none | (short & (at > K // 2)), -1).to(torch.int32)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    s["targets"] = t.masked_fill(torch.rand(T, generator=g, device="cuda") < 0.1, -100) if c["hard"] else None
    if c["train"]:
        s["dkl"] = torch.rand(T, generator=g, device="cuda") / T
        s["dlogp"] = -torch.rand(T, generator=g, device="cuda") / T if c["hard"] else None
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"qkrope": _qkrope_own, "cross": _cross_own, "distill": _distill_own}[op](state)
    return {"qkrope": _qkrope_plain, "cross": _cross_plain, "distill": _distill_plain}[op](state)


def _qkrope_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    r = M.QkRope(inv_freq=s["inv_freq"], pos=s["pos"], axis=s["axis"], interleaved=c["inter"], norm=c["norm"], w_q=s["w_q"],
                 w_k=s["w_k"], eps=1e-6, w_offset=c["offset"])
    fw = M.qkrope_fwd(s["q"], s["k"], r)
    out = {"q": fw["q"], "k": fw["k"]}
    if c["train"]:
        bw = M.qkrope_bwd(s["q"], s["k"], s["dq"], s["dk"], r, ws=s.get("ws"))
        s["ws"] = bw.pop("ws")
        out["grads"] = {k: t for k, t in bw.items() if t is not None}
    return out


def _pairs_of(x, rot, inter):
    """The rotated dims of the last axis as (first, second) of each pair, and the others."""
    a = x[..., :rot]
    a = (a[..., 0::2], a[..., 1::2]) if inter else (a[..., :rot // 2], a[..., rot // 2:])
    return a[0], a[1], x[..., rot:]


def _unpair(a, b, rest, inter):
    ab = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _qkrope_plain(s):
    c = s["case"]
    pos = s["pos"] if s["axis"] is None else s["pos"][s["axis"].long()].T
    angle = (pos.double()[:, None] if s["axis"] is None else pos.double()) * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = {}
    grads = {}
    for n, w in (("q", s["w_q"]), ("k", s["w_k"])):
        x = y = s[n].float()
        if c["norm"]:
            w = w.float() + c["offset"]
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            y = x * rstd * w
        a, b, rest = _pairs_of(y, c["rot"], c["inter"])
        out[n] = _unpair(a * cos - b * sin, b * cos + a * sin, rest, c["inter"]).to(torch.bfloat16)
        if c["train"]:
            a, b, rest = _pairs_of(s["d" + n].float(), c["rot"], c["inter"])
            g = _unpair(a * cos + b * sin, b * cos - a * sin, rest, c["inter"])
            if c["norm"]:
                grads["dw_" + n] = (g * (x * rstd)).sum((0, 1))
                g = g * w
                g = rstd * (g - x * (rstd * rstd) * (g * x).mean(-1, keepdim=True))
            grads["d" + n] = g.to(torch.bfloat16)
    if c["train"]:
        out["grads"] = grads
    return out


def _cross_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    a = M.Cross(scale=c["d"] ** -0.5, cap=c["cap"], cu_q=s["cu_q"], cu_k=s["cu_k"], k_len=s["k_len"])
    fw = M.cross_fwd(s["q"], s["k"], s["v"], a, train=c["train"], ws=s.get("ws"))
    s["ws"] = fw["ws"]
    out = {"O": fw["O"], "lse": fw["lse"]}
    if c["train"]:
        out.update(M.cross_bwd(s["q"], s["k"], s["v"], s["dO"], fw, a))
    return out


def _cross_plain(s):
    c = s["case"]
    hq, hk, cap, scale = c["hq"], c["hk"], c["cap"], c["d"] ** -0.5

    def heads(x):  # (T, h, d) -> (hk, h / hk, T, d) fp32
        return x.float().view(x.shape[0], hk, -1, c["d"]).permute(1, 2, 0, 3)

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    S = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    bend = None
    if cap:
        S = S.div_(cap).tanh_()
        bend = 1 - S * S if c["train"] else None
        S = S.mul_(cap)
    if s["cu_q"] is not None:
        i, j = torch.arange(c["Tq"], device="cuda"), torch.arange(c["Tk"], device="cuda")
        doc_i = torch.searchsorted(s["cu_q"], i, right=True, out_int32=True) - 1
        doc_j = torch.searchsorted(s["cu_k"], j, right=True, out_int32=True) - 1
        if s["k_len"] is not None:
            doc_j = doc_j.masked_fill(j - s["cu_k"][doc_j] >= s["k_len"][doc_j], -1)
        S = S.masked_fill_(doc_i[:, None] != doc_j[None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    P = P.div_(l)

    def tokens(x):  # (hk, n, T, d) -> (T, hk n, d) bf16
        return x.permute(2, 0, 1, 3).reshape(x.shape[2], -1, c["d"]).to(torch.bfloat16)

    O = torch.matmul(P, v)
    out = {"O": tokens(O), "lse": (m + l.log()).view(hq, c["Tq"])}
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


def _distill_own(s):
    from bwd_lora_mlp_gb300 import layer as M
    c = s["case"]
    t = M.Teacher(ids=s["ids"], values=s["teacher"], rest=c["rest"])
    fw = M.distill_fwd(s["logits"], t, targets=s["targets"], scale=c["scale"])
    out = {n: fw[n] for n in ("kl", "lse") + (("logp",) if c["hard"] else ())}
    if c["train"]:
        out["dlogits"] = M.distill_bwd(s["logits"], t, fw, s["dkl"], targets=s["targets"], dlogp=s["dlogp"],
                                       scale=c["scale"])["dlogits"]
    return out


def _distill_plain(s):
    c = s["case"]
    ids = s["ids"].long()
    has = ids >= 0
    at = ids.clamp(min=0)
    z = s["logits"].float()
    x = z * c["scale"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    logq = x.gather(1, at) - m - total.log()
    y = (s["teacher"] if c["rest"] else s["teacher"] * c["scale"]).masked_fill(~has, -math.inf)
    if not c["rest"]:
        top = y.amax(-1, keepdim=True)
        y = y - torch.where(top == -math.inf, torch.zeros_like(top), top)
        y = y - y.exp().sum(-1, keepdim=True).clamp(min=1e-30).log()
    p = y.exp()
    mass = p.sum(-1, keepdim=True)
    kl = (p * torch.where(has, y - logq, torch.zeros_like(y))).sum(-1)
    if c["rest"]:
        left = (1 - mass).clamp(min=0)
        mass = mass + left
        spare = at.masked_fill(~has, c["V"])  # (entries that are none go to a column of their own)
        others = torch.cat((e, torch.zeros_like(m)), -1).scatter_(1, spare, 0.0)[:, :-1].sum(-1, keepdim=True)
        ratio = left / others * total  # p over q of what is left
        kl = kl + torch.where(left > 0, left * ratio.clamp(min=1e-30).log(), torch.zeros_like(left)).squeeze(1)
    out = {"kl": kl, "lse": lse.squeeze(1)}
    if c["hard"]:
        lse1 = lse if c["scale"] == 1 else z.logsumexp(-1, keepdim=True)
        t = s["targets"]
        hit = (t >= 0)[:, None]
        col = t.clamp(min=0)[:, None]
        out["logp"] = torch.where(hit, z.gather(1, col) - lse1, torch.zeros_like(m)).squeeze(1)
    if c["train"]:
        q = e / total
        w = (s["dkl"] * c["scale"])[:, None]
        if c["rest"]:
            d = w * q * (mass - ratio)
            fix = torch.where(has, w * (q.gather(1, at) * ratio - p), torch.zeros_like(p))
        else:
            d = w * mass * q
            fix = -w * p
        d.scatter_add_(1, at, fix)
        if c["hard"]:
            h = torch.where(hit, s["dlogp"][:, None], torch.zeros_like(m))
            d -= h * (z - lse1).exp()
            d.scatter_add_(1, col, h)
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, gradients by differentiation of the forward


def exact(case, seed):
    s = prepare(case, seed)
    return {"qkrope": _qkrope_exact, "cross": _cross_exact, "distill": _distill_exact}[case["op"]](case, s)


def _qkrope_exact(c, s):
    r = c["rot"] // 2
    i = torch.arange(r, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["inter"] else (i, i + r)
    pos = s["pos"].double().view(c["axes"], -1)
    axis = torch.zeros_like(i) if s["axis"] is None else s["axis"].long()
    turn = torch.polar(torch.ones(c["T"], r, dtype=torch.float64, device="cuda"), pos[axis].T * s["inv_freq"].double())
    out, leaves, names, ups = {}, [], [], []
    for n in ("q", "k"):
        x = s[n].double().requires_grad_(c["train"])
        leaves, names = leaves + [x], names + ["d" + n]
        y = x
        if c["norm"]:
            w = s["w_" + n].double().requires_grad_(c["train"])
            leaves, names = leaves + [w], names + ["dw_" + n]
            y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + 1e-6) * (w + c["offset"])
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        full = y.clone()
        full[..., first], full[..., second] = z.real, z.imag
        out[n] = full
        ups.append(s["d" + n].double() if c["train"] else None)
    if c["train"]:
        got = torch.autograd.grad((out["q"], out["k"]), leaves, ups)
        out["grads"] = dict(zip(names, got))
    return {n: t.detach() if isinstance(t, torch.Tensor) else t for n, t in out.items()}


def _cross_exact(c, s):
    hq, hk = c["hq"], c["hk"]
    n, scale = hq // hk, 1 / math.sqrt(c["d"])
    cu_q, cu_k, lens = _segments(c)
    O = torch.zeros(c["Tq"], hq, c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, c["Tq"], dtype=torch.float64, device="cuda")
    grads = {"dQ": torch.zeros_like(O)}
    for name in ("dK", "dV"):
        grads[name] = torch.zeros(c["Tk"], hk, c["d"], dtype=torch.float64, device="cuda")
    for q0, q1, k0, m in zip(cu_q, cu_q[1:], cu_k, lens):
        for g in range(hk):
            q = s["q"][q0:q1, g * n:(g + 1) * n].double().requires_grad_(c["train"])
            k, v = (s[x][k0:k0 + m, g].double().requires_grad_(c["train"]) for x in ("k", "v"))
            z = torch.einsum("ihd,jd->hij", q, k) * scale
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            o = torch.einsum("hij,jd->ihd", torch.softmax(z, -1), v)
            O[q0:q1, g * n:(g + 1) * n] = o.detach()
            lse[g * n:(g + 1) * n, q0:q1] = torch.logsumexp(z.detach(), -1)
            if c["train"]:
                dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dO"][q0:q1, g * n:(g + 1) * n].double())
                grads["dQ"][q0:q1, g * n:(g + 1) * n] = dq
                grads["dK"][k0:k0 + m, g] = dk
                grads["dV"][k0:k0 + m, g] = dv
            del z, o
    return {"O": O, "lse": lse, **(grads if c["train"] else {})}


def _distill_exact(c, s):
    if c["T"] * c["V"] > 1 << 30:
        return None
    z = s["logits"].double().requires_grad_(c["train"])
    ls = torch.log_softmax(z * c["scale"], -1)
    has = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    some = has.any(-1)
    y = s["teacher"].double()
    if not c["rest"]:
        y = torch.log_softmax((y * c["scale"]).masked_fill(~has, -1e300), -1)
    p = torch.where(has & some[:, None], y.exp(), torch.zeros_like(y))
    kl = (p * (y - ls.gather(1, at))).sum(-1)
    if c["rest"]:
        seen = torch.zeros_like(ls, dtype=torch.int32).scatter_add_(1, at, has.int()) > 0
        left = (1 - p.sum(-1)).clamp(min=0)
        others = torch.logsumexp(ls.masked_fill(seen, -math.inf), -1)
        kl = kl + torch.where(left > 0, left * (left.clamp(min=1e-300).log() - others), torch.zeros_like(left))
    out = {"kl": kl, "lse": torch.logsumexp(z.detach() * c["scale"], -1)}
    if c["hard"]:
        t = s["targets"]
        l1 = torch.log_softmax(z, -1).gather(1, t.clamp(min=0)[:, None]).squeeze(1)
        out["logp"] = torch.where(t < 0, torch.zeros_like(l1), l1)
    if c["train"]:
        ends = [out["kl"]] + ([out["logp"]] if c["hard"] else [])
        ups = [s["dkl"].double()] + ([s["dlogp"].double()] if c["hard"] else [])
        out["dlogits"], = torch.autograd.grad(ends, z, ups)
    return {n: t.detach() for n, t in out.items()}
