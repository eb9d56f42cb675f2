"""distill_bwd at the teacher's tokens of rows whose divergence has no gradient (dkl of 0, or none given), while their own
log probability has one, against the fp64 definition.

Tolerance: a gradient is a difference of parts of at most |dlogp| (and scale |dkl|), each off by 2^-16 of itself
(a probability's logarithm is off by less than 2^-17), rounded once more to bf16: 2^-8 of itself."""
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


def _inputs(T, V, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * 2.5).to(dtype)
    lp, ids = torch.log_softmax(z.float() + torch.randn(T, V, generator=g), -1).topk(K, -1)
    return z.cuda(), ids.to(torch.int32).cuda(), lp.cuda()


def _compare(z, ids, v, t, dkl, dlogp, scale, rest):
    teacher = M.Teacher(ids, v, rest)
    fw = M.distill_fwd(z, teacher, t, scale)
    got = M.distill_bwd(z, teacher, fw, dkl, t, dlogp, scale)["dlogits"]
    want = O.distill_backward(host64(z), ids.cpu().numpy(), host64(v), None if dkl is None else host64(dkl), t.cpu().numpy(),
                              host64(dlogp), scale, rest)
    parts = np.abs(host64(dlogp)) + (0 if dkl is None else scale * np.abs(host64(dkl)))
    half = 0.0 if z.dtype == torch.float32 else 2.0 ** -8
    assert torch.isfinite(got).all()
    off = np.abs(host64(got) - want)
    assert (off <= half * np.abs(want) + 2.0 ** -16 * parts[:, None]).all(), off.max()


@pytest.mark.parametrize("scale", [1.0, 0.7, 1.5])
@pytest.mark.parametrize("low", [-float("inf"), "lowest", -1e4, -100.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V", [300, 20011])
def test_masked_rows_whose_divergence_has_no_gradient(V, rest, given, dtype, low, scale):
    """The teacher's tokens hold all that the mask leaves, some of it, or none; the row's own token is one of them or not."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    T, K = 12, 6
    z, ids, v = _inputs(T, V, K, dtype)
    for t in range(0, T, 3):  # nothing but the entries; nothing but two of them; (none masked)
        keep = ids[t].long()
        row = z[t].clone()
        z[t] = low
        z[t, keep] = row[keep]
        z[t + 1, ids[t + 1, 2:].long()] = low
    z[10] = low
    t = ids[:, 0].clone()
    t[3], t[4], t[5] = (int(ids[3, 1]) + 1) % V, ids[4, 5], (int(ids[5, 0]) + 1) % V
    t[6] = -100
    g = torch.Generator().manual_seed(1)
    dlogp = torch.randn(T, generator=g).cuda()
    dlogp[8] = 0
    dkl = None
    if given:
        dkl = torch.randn(T, generator=g).cuda()
        dkl[:7] = 0
    _compare(z, ids, v, t, dkl, dlogp, scale, rest)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("scale", [1.0, 0.8])
def test_entries_that_hold_nearly_all(scale, given):
    """Entries that lie 30, 100 and 300 above the others: the others' share of a row's sum is down to nothing."""
    z, ids, v = _inputs(9, 4000, 4, torch.float32)
    for i, up in enumerate((30.0, 100.0, 300.0)):
        rows = slice(3 * i, 3 * i + 3)
        z[rows].scatter_(1, ids[rows].long(), up + torch.tensor([2.0, 0.0, -1.0, 1.0], device="cuda").expand(3, 4).contiguous())
    t = ids[:, 1].clone()
    t[::3] = 7
    dlogp = torch.linspace(-1, 1.5, 9, device="cuda")
    _compare(z, ids, v, t, torch.zeros(9, device="cuda") if given else None, dlogp, scale, True)


def test_a_teacher_that_is_nan_counts_nothing_where_the_divergence_has_no_gradient():
    z, ids, v = _inputs(4, 500, 5, torch.bfloat16)
    t = torch.tensor([3, 9, 2, 70], dtype=torch.int32, device="cuda")
    dlogp = torch.tensor([1.0, -1.0, 0.5, 2.0], device="cuda")
    for rest in (False, True):
        want = None
        for bad in (None, float("nan"), float("inf")):
            w = v.clone()
            if bad is not None:
                w[1, 2] = bad
            teacher = M.Teacher(ids, w, rest)
            got = M.distill_bwd(z, teacher, M.distill_fwd(z, teacher, t), None, t, dlogp)["dlogits"]
            want = got if bad is None else want
            assert torch.isfinite(got).all() and torch.equal(got, want)
