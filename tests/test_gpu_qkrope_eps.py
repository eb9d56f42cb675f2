"""Norms of heads of zeros and of tiny values under the smallest eps that qkrope takes, against the fp64 definition
(tolerances as for other heads: 2^-8 of a bf16 result, and before it 2^-17 of the head's largest value; dw, fp32, 1e-5 of
its largest, where the terms are of one size)."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _near(name, got, want):
    got = host64(got)
    assert np.isfinite(got).all(), name
    off = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - 2.0 ** -17 * np.abs(want).max(axis=-1, keepdims=True)
    assert (off <= 0).all(), (name, float(off.max()))


@pytest.mark.parametrize("d", [128, 72])
@pytest.mark.parametrize("tiny", [0.0, 1e-19, 1e-10])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-6])
def test_small_heads_and_the_smallest_eps(eps, tiny, d):
    T, hq = 21, 6
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(T, hq, d, generator=g) * tiny).bfloat16().cuda()
    dq = (torch.randn(T, hq, d, generator=g) * 64).bfloat16().cuda()
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    f = (1e4 ** (-torch.arange(d // 2).double() / (d // 2))).float().cuda()
    r = M.QkRope(inv_freq=f, norm=True, w_q=w, eps=eps)
    kw = dict(angles=O.qkrope_angles(T, f.cpu().numpy()), norm=True, w=host64(w), eps=float(np.float32(eps)))
    _near("q", M.qkrope_fwd(q, None, r)["q"], O.qkrope_forward(host64(q), **kw))
    bw = M.qkrope_bwd(q, None, dq, None, r)
    dx, dw = O.qkrope_backward(host64(q), host64(dq), **kw)
    _near("dq", bw["dq"], dx)
    assert np.abs(host64(bw["dw_q"]) - dw).max() <= 1e-5 * np.abs(dw).max()
