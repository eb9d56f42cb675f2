"""Residual add with norms (addnorm_fwd, addnorm_bwd) against the fp64 definition.

Tolerances.  All arithmetic is fp32 from exact inputs, one rounding at the end: bf16 outputs are within
2^-8 of the exact value (relative, each element) plus the fp32 error; fp32 outputs and the sums over
tokens within 1e-5 in the Frobenius norm (a few hundred fp32 roundings, partly averaging)."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import check, host64

pytestmark = pytest.mark.gpu

BF16_REL = 2.0 ** -8 + 1e-5
F32_REL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _rand(shape, seed, std=1.0, mean=0.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def _case(T, d, post, gate, inn, h32, w32, add=True, seed=0):
    hd, wd = (torch.float32 if h32 else torch.bfloat16), (torch.float32 if w32 else torch.bfloat16)
    x = {"h": _rand((T, d), seed, 2.0, 0.3, hd), "y": _rand((T, d), seed + 1, 0.5) if add else None,
         "dh_out": _rand((T, d), seed + 2, 0.1, 0.0, hd), "dx": _rand((T, d), seed + 3, 0.1) if inn else None,
         "w_in": _rand((d,), seed + 4, 0.2, 1.0, wd) if inn else None,
         "w_post": _rand((d,), seed + 5, 0.2, 1.0, wd) if post else None,
         "gate": _rand((d,), seed + 6, 0.5, 0.0, wd) if gate else None}
    return x


def _run(x, alpha, off, weights=True, stream=None, dh_out=True):
    c = {k: None if v is None else v.cuda() for k, v in x.items()}
    n = M.AddNorm(c["w_in"], c["w_post"], c["gate"], alpha, 1e-5, off)
    fw = M.addnorm_fwd(c["h"], c["y"], n, stream=stream)
    bw = M.addnorm_bwd(c["h"], c["y"], c["dh_out"] if dh_out else None, c["dx"], fw, n, weights=weights, stream=stream)
    return fw, bw


def _ref(x, alpha, off, dh_out=True):
    f = {k: None if v is None else v.double().numpy() for k, v in x.items()}
    par = dict(w_in=f["w_in"], w_post=f["w_post"], gate=f["gate"], alpha=alpha, eps=1e-5, w_offset=off)
    return (O.addnorm_forward(f["h"], f["y"], **par),
            O.addnorm_backward(f["h"], f["y"], f["dh_out"] if dh_out else None, f["dx"], **par))


def _compare(got, ref):
    for n, t in got.items():
        if n == "ws":
            continue
        assert (t is None) == (ref[n] is None), n
        if t is not None:
            check(n, host64(t), ref[n], BF16_REL if t.dtype == torch.bfloat16 else F32_REL)


FORMS = [(True, True, True), (False, False, True), (True, False, False), (False, True, True), (False, True, False)]


@pytest.mark.parametrize("T,d", [(1, 32), (3, 4096), (17, 96), (130, 1056), (700, 256), (9, 16384), (33, 8224)])
@pytest.mark.parametrize("h32,w32", [(False, False), (True, False), (False, True), (True, True)])
def test_against_the_definition(T, d, h32, w32):
    for i, (post, gate, inn) in enumerate(FORMS):
        x = _case(T, d, post, gate, inn, h32, w32, seed=T + d + 10 * i)
        alpha, off = (0.5, 1.0) if i % 2 else (1.0, 0.0)
        (fw, bw), (rf, rb) = _run(x, alpha, off), _ref(x, alpha, off)
        _compare(fw, rf)
        _compare(bw, rb)


@pytest.mark.parametrize("h32", [False, True])
def test_norm_alone(h32):
    x = _case(50, 320, False, False, True, h32, False, add=False, seed=3)
    (fw, bw), (rf, rb) = _run(x, 1.0, 0.0), _ref(x, 1.0, 0.0)
    assert torch.equal(fw["h"].cpu(), x["h"])
    _compare({k: v for k, v in fw.items() if k != "h"}, rf)
    _compare(bw, rb)


def test_without_the_streams_gradient():
    x = _case(40, 512, True, True, True, False, False, seed=5)
    (_, bw), (_, rb) = _run(x, 0.7, 0.0, dh_out=False), _ref(x, 0.7, 0.0, dh_out=False)
    _compare(bw, rb)


def test_frozen_weights_leave_the_rest_as_it_is():
    x = _case(300, 1024, True, True, True, False, False, seed=6)
    (_, all_), (_, some) = _run(x, 0.7, 0.0), _run(x, 0.7, 0.0, weights=False)
    assert some["dw_in"] is None and some["dw_post"] is None and some["dgate"] is None
    assert torch.equal(all_["dh"], some["dh"]) and torch.equal(all_["dy"], some["dy"])


def test_rows_of_zeros_and_of_large_values():
    x = _case(4, 256, True, False, True, True, False, seed=8)
    x["h"][0] = 0
    x["y"][0] = 0
    x["h"][1] *= 1e15
    x["y"][2] = x["y"][2] * 1e15
    (fw, bw), (rf, rb) = _run(x, 1.0, 0.0), _ref(x, 1.0, 0.0)
    for i in range(4):  # each row by itself: their sizes differ by 15 orders of magnitude
        check("h", host64(fw["h"])[i], rf["h"][i], F32_REL)
        check("x", host64(fw["x"])[i], rf["x"][i], BF16_REL)
        check("dy", host64(bw["dy"])[i], rb["dy"][i], BF16_REL)
        check("dh", host64(bw["dh"])[i], rb["dh"][i], F32_REL)


def test_no_tokens():
    x = _case(0, 64, True, True, True, False, False)
    fw, bw = _run(x, 1.0, 0.0)
    assert fw["x"].shape == (0, 64)
    for n in ("dw_in", "dw_post", "dgate"):
        assert torch.all(bw[n] == 0), n


def test_same_bits_again_and_on_a_side_stream():
    x = _case(999, 2080, True, True, True, False, False, seed=12)
    want = _run(x, 0.5, 0.0)
    side = torch.cuda.Stream()
    for stream in (None, side):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            got = _run(x, 0.5, 0.0, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for n in a:
                if n != "ws" and a[n] is not None:
                    assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    x = _case(64, 512, True, True, True, True, True, seed=15)
    _, bw = _run(x, 0.5, 0.0)

    def f(x):
        n = M.AddNorm(x["w_in"].cuda(), x["w_post"].cuda(), x["gate"].cuda(), 0.5, 1e-5, 0.0)
        fw = M.addnorm_fwd(x["h"].cuda(), x["y"].cuda(), n)
        return ((fw["h"].double().cpu() * x["dh_out"].double()).sum()
                + (fw["x"].double().cpu() * x["dx"].double()).sum()).item()

    for name, src in (("dh", "h"), ("dw_in", "w_in"), ("dw_post", "w_post"), ("dgate", "gate")):
        step = torch.sign(bw[name].float().cpu()) * 0.05
        up, dn = dict(x), dict(x)
        up[src], dn[src] = x[src] + step, x[src] - step
        said = (bw[name].double().cpu() * (up[src] - dn[src]).double()).sum().item()
        seen = f(up) - f(dn)
        assert abs(seen - said) <= 0.03 * abs(said), (name, seen, said)  # x is rounded to bf16 in both forwards


def test_offsets_past_32_bits():
    """140000 tokens of 16384: 2.3e9 elements a tensor; rows from both ends against the definition."""
    T, d = 140000, 16384
    g = torch.Generator(device="cuda").manual_seed(2)
    h, y = (torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.randn(d, generator=g, device="cuda", dtype=torch.bfloat16)
    n = M.AddNorm(w, w, None, 0.5)
    fw = M.addnorm_fwd(h, y, n)
    bw = M.addnorm_bwd(h, y, y, h, fw, n)
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    f = [t[rows].double().cpu().numpy() for t in (h, y)]
    wn = w.double().cpu().numpy()
    rf = O.addnorm_forward(*f, wn, wn, None, 0.5)
    rb = O.addnorm_backward(*f, f[1], f[0], wn, wn, None, 0.5)
    for name, got, ref in (("h", fw, rf), ("x", fw, rf), ("dh", bw, rb), ("dy", bw, rb)):
        check(name, host64(got[name][rows]), ref[name], BF16_REL)
    del h, y, fw, bw
    torch.cuda.empty_cache()
