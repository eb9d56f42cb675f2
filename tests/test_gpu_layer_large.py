"""The largest sizes of qkrope, cross attention and distillation that a test can afford, and calls at once: lists of key
tiles that are full, tokens by the million, rows of millions of logits, calls on several streams beside each other.

References are the definitions in 64 bits, formed on the GPU where the host would take minutes; tolerances are those of
the operators' own tests."""
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


def _bf(*shape, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


@pytest.mark.parametrize("docs", [False, True])
@pytest.mark.parametrize("heads", [76, 1])  # (76: two CTAs share a head's 8192 tiles; 1: 152)
def test_a_query_of_a_million_states(heads, docs):
    Tk, d, used = 2 ** 20 - 3, 8, 2 ** 20 - 4000
    q, k, v = _bf(2, heads, d, seed=1, std=3.0), _bf(Tk, heads, d, seed=2), _bf(Tk, heads, d, seed=3)
    a = M.Cross(d ** -0.5)
    if docs:  # the first query sees `used` states, the second none of the others
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        a = M.Cross(d ** -0.5, cu_q=i32(0, 1, 2), cu_k=i32(0, Tk - 900, Tk), k_len=i32(used, 0))
        v[used:] = float("nan")
    fw = M.cross_fwd(q, k, v, a)
    L.lm_workspace_check(fw["ws"])
    n = used if docs else Tk
    for h in range(0, heads, 25):
        z = (q[:, h].double() @ k[:n, h].double().T) * d ** -0.5
        check("O", host64(fw["O"][:1, h]), (torch.softmax(z, -1) @ v[:n, h].double()).cpu().numpy()[:1], REL)
        # (a million terms: lse is off by a few 2^-24 of 20)
        assert abs(float(fw["lse"][h, 0]) - float(torch.logsumexp(z[0], -1))) <= 2e-5
    if docs:
        assert not fw["O"][1].any() and torch.isneginf(fw["lse"][:, 1]).all()


def test_tokens_by_the_million():
    T = 3_000_001
    q = _bf(T, 1, 8, seed=4)
    f = torch.tensor([1.0, 0.1, 0.01, 0.001], device="cuda")
    got = M.qkrope_fwd(q, None, M.QkRope(inv_freq=f, norm=True))["q"]
    at = torch.tensor([0, 1, 2_432_000, T - 2, T - 1])
    angles = at.double().numpy()[:, None] * f.double().cpu().numpy()
    want = O.qkrope_forward(host64(q[at]), angles, norm=True)
    off = np.abs(host64(got[at]) - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -18 * np.abs(want).max(-1, keepdims=True)
    assert (off <= 1e-30).all()
    # every token's heads keep their length (the norm makes it sqrt 8, a rotation leaves it)
    length = got.double().square().sum(-1)
    assert float((length - 8).abs().max()) <= 8 * 2 * 2.0 ** -8 + 8 * 1e-3  # (bf16; eps beside a small mean square)


@pytest.mark.parametrize("f32", [False, True])
def test_rows_of_millions_of_logits(f32):
    T, V, K = 2, 2 ** 23 + 5, 128
    z = _bf(T, V, seed=5, std=2.0)
    z = z.float() if f32 else z
    teacher = z.float() + _bf(T, V, seed=6).float()
    top, ids = teacher.topk(K, -1)
    lp = top - teacher.logsumexp(-1, keepdim=True)
    t = M.Teacher(ids, lp, rest=True)
    dkl = torch.tensor([1.0, -0.5], device="cuda")
    fw = M.distill_fwd(z, t)
    got = M.distill_bwd(z, t, fw, dkl)["dlogits"]
    x = z.double().requires_grad_()
    ls = torch.log_softmax(x, -1)
    p = lp.double().exp()
    mine = torch.zeros_like(ls, dtype=torch.bool).scatter_(1, ids, True)
    left = 1 - p.sum(-1)
    kl = (p * (lp.double() - ls.gather(1, ids))).sum(-1) + left * (left.log() - torch.logsumexp(ls.masked_fill(mine, -float("inf")), -1))
    want, = torch.autograd.grad(kl, x, dkl.double())
    assert float((fw["kl"].double() - kl).abs().max()) <= 2.0 ** -16
    off = (got.double() - want).abs() - (0 if f32 else 2.0 ** -8) * want.abs() - 2.0 ** -16 * dkl.double().abs()[:, None]
    assert float(off.max()) <= 0
    # (an element of the tail is coef times its share: each off by 2^-16 of itself, and coef by 2^-22 of its parts)
    tail = ~mine
    rel = (got.double() - want).abs()[tail] - ((0 if f32 else 2.0 ** -8) + 2.0 ** -14) * want.abs()[tail]
    assert float(rel.max()) <= 1e-30


def test_calls_on_several_streams_at_once():
    """Each with its own buffers and workspace; and one after the other on two streams with one workspace."""
    q, k, v, dO = _bf(90, 8, 64, seed=1, std=2.0), _bf(1000, 2, 64, seed=2), _bf(1000, 2, 64, seed=3), _bf(90, 8, 64, seed=4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    a = M.Cross(0.125, cu_q=i32(0, 30, 90), cu_k=i32(0, 400, 1000), k_len=i32(300, 600))
    r = M.QkRope(inv_freq=torch.rand(32, device="cuda"), norm=True, w_q=torch.ones(64, device="cuda"))
    z, ids = _bf(90, 5000, seed=5), torch.randint(5000, (90, 7), device="cuda")
    t = M.Teacher(ids, _bf(90, 7, seed=6))

    def step(ws=None):
        rot = M.qkrope_fwd(q, None, r)["q"]
        fw = M.cross_fwd(rot, k, v, a, ws=ws)
        bw = M.cross_bwd(rot, k, v, dO, fw, a)
        rb = M.qkrope_bwd(q, None, bw["dQ"], None, r)
        lo = M.distill_fwd(z, t)
        return [fw["O"], fw["lse"], bw["dK"], bw["dV"], rb["dq"], rb["dw_q"], lo["kl"], M.distill_bwd(z, t, lo, lo["kl"])["dlogits"]]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for one in got for x, y in zip(one, want))
    ws = L.workspace(M.cross_workspace_size(90, 1000, 8, 2, 64))
    torch.cuda.synchronize()
    got = []
    for s in (streams[0], streams[1], streams[0]):
        with torch.cuda.stream(s):
            got.append(step(ws))
        streams[0].wait_stream(s)
        streams[1].wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for one in got for x, y in zip(one, want))
    L.lm_workspace_check(ws)
