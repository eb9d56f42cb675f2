"""Rows of logits that several CTAs share (few rows): the same results as rows that one CTA takes alone, call
after call, while other work keeps the SMs busy and a cluster's CTAs start at different times."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 50257), (4, 131072), (90, 50257), (200, 32000)])  # eight, eight, four, two CTAs a row
def test_shared_rows_call_after_call(T, V, dtype):
    """700 rows are taken one CTA each; the same rows in calls of a few are shared.  A sum joined in other
    parts is another rounding: 1e-5, as for the sums themselves; the alternatives are the same."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.randn(700, V, generator=g, device="cuda") * 3).to(dtype)
    t = torch.randint(0, V, (700,), generator=g, device="cuda")
    want = M.logprob_fwd(x, t, 20)
    side, busy = torch.cuda.Stream(), torch.ones(64 << 20, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(40):
            busy.mul_(1.0)
    got = [(a, M.logprob_fwd(x[a:a + T], t[a:a + T], 20)) for a in list(range(0, 700 - T + 1, max(T, 14)))[:50]]
    torch.cuda.synchronize()
    for a, r in got:
        assert torch.equal(r["top_ids"], want["top_ids"][a:a + T])
        for n in ("logp", "lse", "entropy", "top_logp"):
            assert (r[n] - want[n][a:a + T]).abs().max() <= 1e-5, (n, a)
