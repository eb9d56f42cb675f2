"""A NaN logit anywhere in a long row (logprob_fwd, logprob_bwd): the row's lse, entropy, logp and gradient are
NaN, the NaN is the first alternative, and the other rows keep their bits."""
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
@pytest.mark.parametrize("V", [50257, 131072])
@pytest.mark.parametrize("T", [4, 90, 200, 700])  # eight, four, two CTAs a row, one
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_a_nan_in_a_long_row(T, V, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(V + T)
    buf = (torch.randn(T, V + 3, generator=g, device="cuda") * 3).to(dtype)
    x = buf[:, 1:V + 1]  # rows that begin and end off 16 bytes
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[2] = -100
    clean = M.logprob_fwd(x, t, 3, scale)
    ones = torch.ones(T, device="cuda")
    first = M.logprob_bwd(x, t, clean, ones, ones, scale)["dlogits"]
    # the row's first element (before its first 16 bytes) and its last, the first batches, the middle, the last ones
    for j in (0, 5, 300, 9000, V // 2, V - 5000, V - 40, V - 1):
        for row in (1, 2):
            was = x[row, j].item()
            x[row, j] = float("nan")
            fw = M.logprob_fwd(x, t, 3, scale)
            assert torch.isnan(fw["lse"][row]) and torch.isnan(fw["entropy"][row]), (row, j)
            assert torch.isnan(fw["logp"][row]) if row == 1 else fw["logp"][row] == 0, (row, j)
            assert fw["top_ids"][row, 0] == j and torch.isnan(fw["top_logp"][row]).all(), (row, j)
            d = M.logprob_bwd(x, t, fw, ones, ones, scale)["dlogits"]
            assert torch.isnan(d[row]).all(), (row, j)
            keep = torch.arange(T, device="cuda") != row
            for n in ("lse", "entropy", "logp", "top_ids", "top_logp"):
                assert torch.equal(fw[n][keep], clean[n][keep]), (n, row, j)
            assert torch.equal(d[keep], first[keep]), (row, j)
            x[row, j] = was
