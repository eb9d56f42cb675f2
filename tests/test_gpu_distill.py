"""Distillation from a teacher's top logits (distill_fwd, distill_bwd) against the fp64 definition: types,
vocabularies around the vector and CTA sizes, strides, tokens given twice, short and empty rows, masked logits,
entries that hold nearly all of the mass, temperatures, tokens' own loss, captured and on other streams.

Tolerances.  Everything is fp32 until dlogits of bf16 logits is rounded.  A log probability's terms are off by 2^-24 of
themselves each (x = scale z, the maximum, lse): with |x| below 2^5 and a sum of up to 2^17 terms, whose pairwise
parts add fewer than 2^5 roundings, log q is off by less than 2^-17; kl, an average of such, by 2^-16 (and of
its own size 2^-20).  A gradient is a product of probabilities off by 2^-16 of themselves, so by 2^-16 of the
parts that it is the difference of: W q and p, at most the row's factors."""
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


def _inputs(T, V, K, f32=False, rest=False, seed=0, pad=0, off=0, std=2.5, wide=False, v_bf16=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, V, generator=g) * std
    z = z if f32 else z.bfloat16()
    teacher = z.float() + torch.randn(T, V, generator=g)
    k = min(K, V)
    top, ids = teacher.topk(k, -1)
    if rest:
        top = top - teacher.logsumexp(-1, keepdim=True)
    if k < K:
        ids = torch.cat((ids, torch.full((T, K - k), -1)), -1)
        top = torch.cat((top, torch.zeros(T, K - k)), -1)
    full = torch.zeros(T, off + V + pad, dtype=z.dtype).cuda()
    full[:, off:off + V] = z.cuda()
    top = top.bfloat16() if v_bf16 else top
    return full[:, off:off + V], ids.to(torch.int64 if wide else torch.int32).cuda(), top.cuda()


def _check(z, ids, v, targets=None, scale=1.0, rest=False, dlogits=None, seed=1):
    T, V = z.shape
    g = torch.Generator().manual_seed(seed)
    dkl = torch.randn(T, generator=g).cuda()
    dkl[1::5] = 0
    dlogp = torch.randn(T, generator=g).cuda() if targets is not None else None
    z64, ids_h, v_h = host64(z), ids.cpu().numpy(), host64(v)
    t_h = None if targets is None else targets.cpu().numpy()
    teacher = M.Teacher(ids, v, rest)
    fw = M.distill_fwd(z, teacher, targets, scale)
    want = O.distill_forward(z64, ids_h, v_h, t_h, scale, rest)
    for n in ("kl", "lse", "logp"):
        if want[n] is None:
            assert fw[n] is None
            continue
        got, ref = host64(fw[n]), want[n]
        fin = np.isfinite(ref)
        assert np.array_equal(got[~fin], ref[~fin]), n
        assert (np.abs(got[fin] - ref[fin]) <= 2.0 ** -16 + 2.0 ** -20 * np.abs(ref[fin])).all(), \
            (n, np.abs(got[fin] - ref[fin]).max())
    d64 = O.distill_backward(z64, ids_h, v_h, host64(dkl), t_h, None if dlogp is None else host64(dlogp), scale, rest)
    got = M.distill_bwd(z, teacher, fw, dkl, targets, dlogp, scale, dlogits)["dlogits"]
    parts = scale * np.abs(host64(dkl)) + (0 if dlogp is None else np.abs(host64(dlogp)))
    # (an element's parts are at most the row's factors; far smaller where its own probability is, by which their errors go)
    off = np.abs(host64(got) - d64)
    half = 0.0 if z.dtype == torch.float32 else 2.0 ** -8
    assert (off <= half * np.abs(d64) + 2.0 ** -16 * parts[:, None]).all(), off.max()
    q = np.exp(scale * (z64 - z64.max(1, keepdims=True)))
    q = q / q.sum(1, keepdims=True)
    small = np.isfinite(q) & (q < 1e-3)
    if rest is False and targets is None and small.any():  # elsewhere the gradient is W q alone: its own relative error
        np.put_along_axis(small, np.clip(ids_h, 0, V - 1).astype(np.int64), False, axis=1)
        assert (off <= (half + 2.0 ** -15) * np.abs(d64) + 1e-30)[small].all()
    return teacher, fw, dkl, dlogp, got


SIZES = [(1, 1, 1), (3, 7, 3), (5, 8, 8), (4, 63, 20), (9, 300, 64), (7, 2049, 128), (3, 16384 + 9, 5), (160, 1000, 32),
         (700, 515, 10)]


@pytest.mark.parametrize("T,V,K", SIZES)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_against_the_definition(T, V, K, rest, f32):
    z, ids, v = _inputs(T, V, K, f32, rest)
    _check(z, ids, v, rest=rest)


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.7])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("f32,wide,v_bf16", [(False, True, False), (True, False, True)])
def test_temperatures_and_the_tokens_own_loss(scale, rest, f32, wide, v_bf16):
    T, V = 33, 777
    z, ids, v = _inputs(T, V, 20, f32, rest, wide=wide, v_bf16=v_bf16)
    t = torch.randint(V, (T,), generator=torch.Generator().manual_seed(3)).to(torch.int64 if wide else torch.int32).cuda()
    t[::4], t[1], t[2] = ids[::4, 0].to(t.dtype), -100, V  # (some are entries, some none)
    _check(z, ids, v, t, scale, rest)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V,cluster", [(150001, 8), (70000, 8), (33333, 4)])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_of_several_ctas(V, cluster, f32, rest):
    """Few long rows, each shared by a cluster; more vectors than bytes in shared memory only where a CTA has a row."""
    z, ids, v = _inputs(3, V, 64, f32, rest)
    ids[0, :4] = torch.tensor([0, V - 1, V // 2, 1], device="cuda")
    _check(z, ids, v, rest=rest, targets=torch.tensor([0, V - 1, 5], device="cuda"))


def test_more_vectors_than_bytes_that_mark_them():
    """One CTA a row (many rows), longer than what each vector has a byte for."""
    T, V = 320, 4 * 16384 + 1003
    z, ids, v = _inputs(T, V, 40, True, True)
    g = torch.Generator().manual_seed(5)
    some = torch.randint(T, (4,), generator=g).tolist()
    fw = M.distill_fwd(z, M.Teacher(ids, v, True))
    assert T * 2 > 152 * 4  # (no cluster)
    want = O.distill_forward(host64(z[some]), ids[some].cpu().numpy(), host64(v[some]), rest=True)
    assert np.abs(host64(fw["kl"][some]) - want["kl"]).max() <= 2.0 ** -16


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad,off", [(7, 0), (64, 0), (3, 5), (5000, 1)])
def test_strides(f32, pad, off):
    z, ids, v = _inputs(37, 1001, 16, f32, True, pad=pad, off=off)
    teacher, fw, dkl, _, got = _check(z, ids, v, rest=True)
    assert (got.data_ptr() - z.data_ptr()) % 16 == 0 and (got.stride(0) - z.stride(0)) * z.element_size() % 16 == 0
    flat = torch.empty(37, 1001, dtype=z.dtype, device="cuda")  # (rows that lie differently)
    M.distill_bwd(z, teacher, fw, dkl, dlogits=flat)
    assert torch.equal(flat, got)
    side = z._base.clone()
    M.distill_bwd(z, teacher, fw, dkl, dlogits=z)
    assert torch.equal(z, got)
    edge = torch.ones(z._base.shape[1], dtype=torch.bool, device="cuda")
    edge[off:off + 1001] = False
    assert torch.equal(z._base[:, edge], side[:, edge])


@pytest.mark.parametrize("rest", [False, True])
def test_tokens_given_twice_and_short_rows(rest):
    z, ids, v = _inputs(12, 500, 8, False, rest)
    ids[0, 3] = ids[0, 0]
    ids[1] = ids[1, 0]
    ids[2, 1:] = -1
    ids[3] = 500
    ids[4] = -100
    ids[5, ::2] = 2 ** 31 - 1
    v[6, 2] = -float("inf")
    v[7] = -float("inf")
    if rest:
        v[1] -= 3
    _check(z, ids, v, rest=rest, targets=torch.arange(12, device="cuda"))


@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_masked_logits(scale):
    """Logits of -inf, of the type's lowest value, whole rows of them; entries on masked tokens."""
    for rest in (False, True):
        for low in (-float("inf"), float(torch.finfo(torch.bfloat16).min), -1e4):
            z, ids, v = _inputs(8, 300, 6, False, rest)
            z[0, 10:] = low
            z[1] = low
            z[2, ids[2, 0].long()] = low
            keep = ids[3].long()
            row = z[3].clone()
            z[3] = low
            z[3, keep] = row[keep]     # nothing but the entries
            z[4, keep[0]] = low
            _check(z, ids, v, rest=rest, scale=scale, targets=torch.full((8,), 5, device="cuda"))


def test_entries_that_hold_nearly_all():
    """What is left has 1e-7 of the mass and less: it comes from its own terms, not from 1 - sum q."""
    z, ids, v = _inputs(6, 4000, 4, True, True, std=1.0)
    z.scatter_(1, ids.long(), torch.tensor([30.0, 28.0, 27.0, 29.0], device="cuda").expand(6, 4).contiguous())
    v.copy_(torch.log_softmax(torch.tensor([3.0, 2.0, 1.0, 1.5, 0.0]), -1)[:4].cuda())
    teacher, fw, dkl, _, got = _check(z, ids, v, rest=True)
    d = O.distill_backward(host64(z), ids.cpu().numpy(), host64(v), host64(dkl), rest=True)
    others = np.ones(d.shape, dtype=bool)
    np.put_along_axis(others, ids.cpu().numpy().astype(np.int64), False, axis=1)
    assert np.allclose(host64(got)[others], d[others], rtol=2.0 ** -14, atol=0)


def test_nan_stays_in_its_row_and_rows_without_gradient_hold_anything():
    z, ids, v = _inputs(6, 700, 5, False, True)
    teacher = M.Teacher(ids, v, True)
    dkl = torch.ones(6, device="cuda")
    dkl[4] = 0
    fw = M.distill_fwd(z, teacher)
    want = M.distill_bwd(z, teacher, fw, dkl)["dlogits"].clone()
    for j in (3, int(ids[2, 1])):
        y = z.clone()
        y[2, j] = float("nan")
        y[4, 11] = float("nan")
        f2 = M.distill_fwd(y, teacher)
        got = M.distill_bwd(y, teacher, f2, dkl)["dlogits"]
        assert f2["kl"][2].isnan() and f2["lse"][2].isnan() and got[2].isnan().all()
        assert not got[4].any() and not want[4].any()
        rows = [0, 1, 3, 5]
        assert torch.equal(f2["kl"][rows], fw["kl"][rows]) and torch.equal(got[rows], want[rows])


def test_against_differences():
    z, ids, v = _inputs(2, 40, 6, True, True)
    dkl = torch.tensor([1.0, -2.0], device="cuda")
    t = torch.tensor([3, 17], device="cuda")
    dlogp = torch.tensor([0.5, 1.5], device="cuda")
    teacher = M.Teacher(ids, v, True)
    fw = M.distill_fwd(z, teacher, t, 0.8)
    d = M.distill_bwd(z, teacher, fw, dkl, t, dlogp, 0.8)["dlogits"]

    def f(z):
        o = O.distill_forward(z, ids.cpu().numpy(), host64(v), t.cpu().numpy(), 0.8, True)
        return (host64(dkl) * o["kl"] + host64(dlogp) * o["logp"]).sum()

    z64 = host64(z)
    for i in range(2):
        for j in range(40):
            e = np.zeros_like(z64)
            e[i, j] = 1e-5
            assert abs((f(z64 + e) - f(z64 - e)) / 2e-5 - float(d[i, j])) < 1e-5


def test_the_same_bits_in_a_graph_on_a_stream_and_beside_each_other():
    z, ids, v = _inputs(50, 3001, 32, False, True)
    t = torch.randint(3001, (50,), device="cuda")
    teacher = M.Teacher(ids, v, True)
    dkl, dlogp = torch.rand(50, device="cuda"), torch.rand(50, device="cuda")

    def step(stream=None):
        fw = M.distill_fwd(z, teacher, t, 0.9, stream=stream)
        return [fw["kl"], fw["logp"], fw["lse"], M.distill_bwd(z, teacher, fw, dkl, t, dlogp, 0.9, stream=stream)["dlogits"]]

    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [step(s) for s in sides for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for one in got for x, y in zip(one, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_no_rows_and_refusals():
    z, ids, v = _inputs(4, 30, 3)
    teacher = M.Teacher(ids, v)
    e = M.distill_fwd(z[:0], M.Teacher(ids[:0], v[:0]))
    assert e["kl"].numel() == 0 and M.distill_bwd(z[:0], M.Teacher(ids[:0], v[:0]), e)["dlogits"].shape == (0, 30)
    fw = M.distill_fwd(z, teacher)
    for call, err in ((lambda: M.distill_bwd(z, teacher, fw, dlogp=fw["kl"], targets=ids[:, 0]), ValueError),
                      (lambda: M.distill_fwd(z, M.Teacher(ids[:, 0], v)), TypeError),
                      (lambda: M.distill_fwd(z, M.Teacher(ids, v[:, :2])), ValueError),
                      (lambda: M.distill_fwd(z, M.Teacher(ids.float(), v)), TypeError),
                      (lambda: M.distill_fwd(z, M.Teacher(ids, v.half())), TypeError),
                      (lambda: M.distill_fwd(z, teacher, scale=0.0), M.LmError),
                      (lambda: M.distill_fwd(z, M.Teacher(torch.zeros(4, 129, dtype=torch.int32, device="cuda"),
                                                          torch.zeros(4, 129, device="cuda"))), M.LmError)):
        with pytest.raises(err):
            call()


def test_offsets_past_32_bits():
    T, V, ld = 3, 1000, 1 << 31
    big = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    z = big.as_strided((T, V), (ld, 1))
    src, ids, v = _inputs(T, V, 9, False, True)
    z.copy_(src)
    _, fw, dkl, _, got = _check(z, ids, v, rest=True)
    M.distill_bwd(z, M.Teacher(ids, v, True), fw, dkl, dlogits=z)
    assert torch.equal(z, got)
