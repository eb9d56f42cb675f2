"""Top alternatives of masked, flat and tied rows (logprob_fwd) against a stable sort: exact indices, the lower first
among equals, in rows of one CTA and shared ones."""
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


def _rows(name, V, dtype, g):
    x = (torch.randn(7, V, generator=g, device="cuda") * 3).to(dtype)
    keep = torch.randperm(V, generator=g, device="cuda")
    masks = {"-inf": -float("inf"), "-1e9": -1e9, "lowest": torch.finfo(dtype).min}
    if name in masks:
        for r, n in enumerate((0, 1, 10, 19, 20, 40, 300)):  # logits that are left
            y = torch.full((V,), masks[name], device="cuda").to(dtype)
            y[keep[:n]] = x[r, keep[:n]]
            x[r] = y
    elif name == "flat":
        for r, c in enumerate((-3.3, 3.3, 0.0, -0.0, 1e-30, -1e4, float("inf"))):
            x[r] = c
    elif name == "low bits":  # fp32 logits that share their upper 16 bits; few of them in bf16
        x = (1 + torch.rand(7, V, generator=g, device="cuda") * 2.0 ** -9).to(dtype)
        x[1::2] *= -1
    elif name == "signed zeros":
        x = torch.where(torch.rand(7, V, generator=g, device="cuda") < 0.5, 0.0, -0.0).to(dtype)
        x[1::2, keep[:5]] = 1
    elif name == "one column of threads":  # the largest of a row lie in few threads
        x[:, ::2048] = x[:, ::2048].abs() + 20
        x[3:, 8::2048] = 30
    else:  # NaN: a few, many, nothing else
        for r, n in enumerate((1, 5, 19, 20, 2000, V // 2, V)):
            x[r, keep[:n]] = float("nan")
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 257, 513, 1023, 1025, 50257, 131072])
@pytest.mark.parametrize("name", ["-inf", "-1e9", "lowest", "flat", "low bits", "signed zeros", "one column of threads", "NaN"])
@pytest.mark.parametrize("copies", [1, 100])  # rows that up to eight CTAs share, and rows of one
def test_alternatives_of_equal_logits(name, V, dtype, copies):
    g = torch.Generator(device="cuda").manual_seed(V)
    if name == "NaN" and V < 2000:
        V = 2000
    if name == "-inf" and V < 300 or name in ("-1e9", "lowest") and V < 300:
        V = 300
    x = _rows(name, V, dtype, g)
    key = torch.nan_to_num(x.double(), nan=float("inf"), posinf=1e300, neginf=-1e300)
    want = torch.sort(key, dim=1, descending=True, stable=True).indices
    x = x.repeat(copies, 1)
    t = torch.zeros(x.shape[0], dtype=torch.int64, device="cuda")
    for k in (1, 20, 32):
        fw = M.logprob_fwd(x, t, k)
        ids = fw["top_ids"].view(copies, 7, k)
        assert torch.equal(ids.long(), want[None, :, :k].expand(copies, 7, k)), k
        top = fw["top_logp"].view(copies, 7, k)
        lp = torch.log_softmax(x[:7].double(), 1).gather(1, want[:, :k])
        fin = torch.isfinite(lp)
        assert ((top[0].double() - lp)[fin].abs() <= 1e-5 + 2.0 ** -23 * x[:7].double().gather(1, want[:, :k])[fin].abs()).all(), k
