"""Calls whose time once was many times that of calls like them.  Times are of a CUDA graph of ten calls, the best of
several replays; the bounds are wide beside what a measurement scatters, and a cliff is far above them."""
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


def _us(call, n=10):
    """Microseconds of one call."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1e3)
    return best


def _attn_step(T, hq, hk, d):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v, dO = (torch.randn(T, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hk, hk, hq))
    a = M.Attn(scale=d ** -0.5)
    fw = M.attn_fwd(q, k, v, a)

    def call():
        M.attn_bwd(q, k, v, dO, M.attn_fwd(q, k, v, a, O=fw["O"], lse=fw["lse"], O_lo=fw["O_lo"], ws=fw["ws"]), a)
    return call


def test_a_last_tile_of_one_token():
    """129 tokens are 256 with less to do: the same tiles, and the tokens past the end come as zeros."""
    part, whole = _us(_attn_step(129, 32, 1, 128)), _us(_attn_step(256, 32, 1, 128))
    assert part <= 1.15 * whole, (part, whole)


@pytest.mark.parametrize("T,V,dtype", [(4, 131072, torch.float32), (4, 131072, torch.bfloat16), (700, 32000, torch.bfloat16),
                                       (700, 32000, torch.float32), (4096, 1000, torch.bfloat16), (4096, 1000, torch.float32)])
@pytest.mark.parametrize("rows", ["ten left of -inf", "ten left of -1e9", "ten left of the lowest value", "flat"])
def test_alternatives_of_masked_and_flat_rows(rows, T, V, dtype):
    """Twenty alternatives where ten logits are not masked, or all are the same negative number, next to rows of
    which each logit is another: not more than three times as long."""
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    fill = {"ten left of -inf": -float("inf"), "ten left of -1e9": -1e9, "ten left of the lowest value": torch.finfo(dtype).min,
            "flat": -3.3}[rows]
    y = torch.full_like(x, fill)
    if rows != "flat":
        at = torch.randperm(V, generator=g, device="cuda")[:10]
        y[:, at] = x[:, at]
    plain, masked = _us(lambda: M.logprob_fwd(x, t, 20)), _us(lambda: M.logprob_fwd(y, t, 20))
    assert masked <= 3 * plain, (masked, plain)
