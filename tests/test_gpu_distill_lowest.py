"""A divergence whose terms fit fp32 although scale times a logit does not: logits of the type's lowest value under a
scale above 1, on which the teacher has little weight.

Tolerance: 2^-20 of kl, and with rest what 1 - sum p is off by (2^-24 of each p and of the sum: below 2^-22) times the
distance of the others, scale times the lowest value at most.  Without rest a value's distance from the row's largest is
rounded, and its product with the scale: 2^-23 of scale times that distance, which is p's relative error and, the
one entry on a masked logit being all of kl, kl's."""
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


@pytest.mark.parametrize("scale", [1.0, 1.6, 4.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("where", ["entries", "others"])
def test_little_weight_on_the_lowest_logits(where, dtype, scale):
    T, V, K = 6, 900, 8
    g = torch.Generator().manual_seed(2)
    low = torch.finfo(dtype).min
    z = torch.randn(T, V, generator=g).to(dtype).cuda()
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]).to(torch.int32).cuda()
    small = torch.tensor([1e-2, 1e-3, 1e-10, 1e-30, 0.05, 0.1])
    p = torch.full((T, K), 0.0) + (1 - small[:, None]) / (K if where == "others" else K - 1)
    if where == "entries":
        p[:, 3] = small / 2
        z.scatter_(1, ids[:, 3:4].long(), low)
    else:
        row = z.gather(1, ids.long())
        z[:] = low
        z.scatter_(1, ids.long(), row)
    v = torch.log(p).cuda()
    got = host64(M.distill_fwd(z, M.Teacher(ids, v, True), scale=scale)["kl"])
    want = O.distill_forward(host64(z), ids.cpu().numpy(), host64(v), scale=scale, rest=True)["kl"]
    fits = want < 3e38
    assert fits.any() and np.isposinf(got[~fits]).all()
    assert (np.abs(got - want)[fits] <= 2.0 ** -20 * want[fits] + (2.0 ** -22 * -low * scale if where == "others" else 0)).all()
    if where == "entries":
        got = host64(M.distill_fwd(z, M.Teacher(ids, v), scale=scale)["kl"])
        want = O.distill_forward(host64(z), ids.cpu().numpy(), host64(v), scale=scale)["kl"]
        fits, far = want < 3e38, scale * host64(v.max(1)[0] - v[:, 3])
        assert fits.any() and np.isposinf(got[~fits]).all()
        assert (np.abs(got - want) <= (2.0 ** -20 + 2.0 ** -23 * far) * want)[fits].all()
