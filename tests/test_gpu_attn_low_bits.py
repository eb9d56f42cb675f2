"""What the rounding of the attention weights leaves out (attn_fwd): multiplied too for rows of few keys and with slopes.

O with O_lo's bits has 16 bits: within 2^-17 of the value, as are weights of two bf16 parts; the exponential, the
sums and the division are a few 2^-23.  Together below 2^-16 in the Frobenius norm.  Weights of one part are rounded
by at most 2^-8 of themselves, 2^-8 / sqrt(3) in the mean square, and a row's errors average like its terms."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _error(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True)])
def test_rows_of_few_keys_and_of_many(d, cap, bias):
    T, hq, hk = 1100, 4, 2
    g = torch.Generator().manual_seed(d)
    q, k, v = ((torch.randn(T, h, d, generator=g) * s).bfloat16() for h, s in ((hq, 2.0), (hk, 1.0), (hk, 1.0)))
    slopes = torch.tensor([2.0 ** -(6 + i) for i in range(hq)])
    a = M.Attn(scale=d ** -0.5, cap=cap, slopes=slopes.cuda() if bias else None)
    fw = M.attn_fwd(q.cuda(), k.cuda(), v.cuda(), a)
    L.lm_workspace_check(fw["ws"])
    got = ((fw["O"].view(torch.int16).int() << 16) + (fw["O_lo"][..., :d].int() << 8)).view(torch.float32).double().cpu().numpy()
    ref = O.attn_forward(*(x.double().numpy() for x in (q, k, v)), O.visible(T), d ** -0.5, cap,
                         slopes.double().numpy() if bias else None)["O"]
    # (capped scores are up to 2^-21 cap off, which moves a weight by as much)
    few = 2.0 ** -16 + cap * 2.0 ** -21
    assert _error(got[:512], ref[:512]) <= few
    assert _error(got[512:], ref[512:]) <= (few if bias else 2.0 ** -8 / 3 ** 0.5)


@pytest.mark.parametrize("lengths", [(511, 300, 200), (1, 2, 3, 64, 129, 400)])
def test_documents_of_few_keys(lengths):
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    T, d = cu[-1], 64
    g = torch.Generator().manual_seed(T)
    q, k, v = ((torch.randn(T, h, d, generator=g) * s).bfloat16() for h, s in ((2, 2.0), (1, 1.0), (1, 1.0)))
    a = M.Attn(scale=d ** -0.5, cu_docs=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    fw = M.attn_fwd(q.cuda(), k.cuda(), v.cuda(), a)
    got = ((fw["O"].view(torch.int16).int() << 16) + (fw["O_lo"].int() << 8)).view(torch.float32).double().cpu().numpy()
    ref = O.attn_forward(*(x.double().numpy() for x in (q, k, v)), O.visible(T, cu_docs=cu), d ** -0.5)["O"]
    assert _error(got, ref) <= 2.0 ** -16
