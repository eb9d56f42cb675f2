"""A teacher's logits far from zero (distill without rest): a softmax does not change when all of a row's logits are
moved together, nor does the divergence from it, whatever the move leaves of fp32.

Tolerance: differences of a row's values are exact in fp32 here or round once, 2^-24 of at most 2^5 scales; with the sums
of up to 128 terms a log probability of the teacher is off by less than 2^-17, and so is the student's: kl by 2^-16
(and 2^-20 of itself), a gradient by 2^-16 of its parts, which are at most scale |dkl|."""
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


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.7])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [0.0, -1e4, 1e4, 3e5, -1e30, "lowest", "largest"])
@pytest.mark.parametrize("K", [1, 7, 128])
def test_rows_of_values_moved_together(K, at, dtype, scale):
    T, V = 9, 700
    g = torch.Generator().manual_seed(K)
    z = torch.randn(T, V, generator=g).cuda() * 2
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]).to(torch.int32).cuda()
    ids[2, K // 2:] = -1
    ends = torch.finfo(dtype)
    v = torch.randn(T, K, generator=g) * 2
    if isinstance(at, str):
        v[:] = ends.min if at == "lowest" else ends.max
        v[1::2, ::2] = 3.0 if at == "lowest" else -3.0  # (masked entries beside others)
    else:
        v += at
    v = v.to(dtype).cuda()
    dkl = torch.randn(T, generator=g).cuda()
    teacher = M.Teacher(ids, v)
    fw = M.distill_fwd(z, teacher, scale=scale)
    want = O.distill_forward(host64(z), ids.cpu().numpy(), host64(v), scale=scale)["kl"]
    off = np.abs(host64(fw["kl"]) - want)
    assert (off <= 2.0 ** -16 + 2.0 ** -20 * np.abs(want)).all(), off.max()
    got = host64(M.distill_bwd(z, teacher, fw, dkl, scale=scale)["dlogits"])
    d = O.distill_backward(host64(z), ids.cpu().numpy(), host64(v), host64(dkl), scale=scale)
    off = np.abs(got - d)
    assert (off <= 2.0 ** -16 * scale * np.abs(host64(dkl))[:, None]).all(), off.max()
