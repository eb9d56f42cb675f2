"""Entropy gradients beyond 1e8 over rows with masked logits (logprob_bwd): a logit without weight has no
gradient, however large the row's is.  Tolerance: fp32 within 1e-5 in the Frobenius norm, as for any gradient."""
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import check, host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


@pytest.mark.parametrize("size", [1.0, 1e10, 1e25])
@pytest.mark.parametrize("skip", [0, 1])  # rows of logits and gradient that lie alike, and not
def test_large_entropy_gradients(size, skip):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(3, 4001, generator=g) * 3).cuda()[:, skip:]
    x[:, ::3] = -float("inf")
    x[1, 1::3] = torch.finfo(torch.float32).min
    x[2, 2::3] = -1e4
    t = torch.tensor([1, -100, 4], device="cuda")
    ge = torch.tensor([1.0, -2.0, 0.5], device="cuda") * size
    gl = torch.ones(3, device="cuda")
    d = M.logprob_bwd(x, t, M.logprob_fwd(x, t), gl, ge)["dlogits"]
    ref = O.logprob_backward(host64(x), t.cpu().numpy(), host64(gl), host64(ge))
    check("dlogits", host64(d), ref, 1e-5)
