"""Norms of query and key heads with the rotation by position (qkrope_fwd, qkrope_bwd) against the fp64
definition: head sizes that are read 16 and 8 bytes at a time, partial rotations, both pairings, axes,
far positions, slices of one buffer, in place, gradients, captured and on other streams.

Tolerances.  A result is rounded to bf16 once: off by 2^-8 of itself at most.  Before it, fp32: cosines and sines off
by 2^-21 and by 2^-30 of a turn, the products and the mean's 2^-24 each: together below 2^-18 of the head's largest
value, 2^-17 for dx, whose two terms each have such errors.  dw is an fp32 sum of up to N terms in chunks, off
by less than 2^-24 sqrt(N) of the terms' 2-norm, 2^-24 N of their sum at most: 1e-5 of the largest
bounds both at these sizes."""
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


def _bf(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16().cuda()


def _near(name, got, want, fp32):
    got = host64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    top = np.abs(want).max(axis=-1, keepdims=True)
    off = np.abs(got - want) - 2.0 ** -8 * np.abs(want) - fp32 * top
    assert (off <= 1e-30).all(), (name, float(off.max()))


def _rope(T, d, rot, inter=False, norm=True, axes=1, far=0, wt=torch.bfloat16, offset=0.0, factor=1.0, wide=False, seed=9):
    """The struct on the device, and what the definition takes (angles, keyword arguments, w_q, w_k)."""
    g = torch.Generator().manual_seed(seed)
    r = M.QkRope(interleaved=inter, factor=factor, norm=norm, w_offset=offset)
    angles = None
    if rot:
        r.inv_freq = (1e4 ** (-torch.arange(rot // 2).double() / (rot // 2))).float().cuda()
        pos = torch.randint(0, 5000, (axes, T) if axes > 1 else (T,), generator=g) + far
        r.pos = pos.to(torch.int64 if wide else torch.int32).cuda()
        if axes > 1:
            r.axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32).cuda()
        angles = O.qkrope_angles(T, r.inv_freq.cpu().numpy(), pos.numpy(), None if axes == 1 else r.axis.cpu().numpy())
    ws = [None, None]
    if norm:
        r.w_q, r.w_k = ((1 - offset + 0.2 * torch.randn(d, generator=g)).to(wt).cuda() for _ in range(2))
        ws = [host64(r.w_q), host64(r.w_k)]
    return r, dict(angles=angles, interleaved=inter, factor=factor, norm=norm, eps=r.eps, w_offset=offset), ws


def _check(T, hq, hk, d, rot, **kw):
    r, o, (wq, wk) = _rope(T, d, rot, **kw)
    q, k, dq, dk = _bf((T, hq, d), 1, 2.0), _bf((T, hk, d), 2, 2.0), _bf((T, hq, d), 3), _bf((T, hk, d), 4)
    fw = M.qkrope_fwd(q, k, r)
    bw = M.qkrope_bwd(q, k, dq, dk, r)
    for n, x, dy, w in (("q", q, dq, wq), ("k", k, dk, wk)):
        _near(n, fw[n], O.qkrope_forward(host64(x), w=w, **o), 2.0 ** -18)
        dx, dw = O.qkrope_backward(host64(x), host64(dy), w=w, **o)
        _near("d" + n, bw["d" + n], dx, 2.0 ** -17)
        if dw is None:
            assert bw["dw_" + n] is None
        else:
            assert np.abs(host64(bw["dw_" + n]) - dw).max() <= 1e-5 * np.abs(dw).max()
    return q, k, dq, dk, r, fw, bw


SHAPES = [(1, 1, 1, 8, 8), (2, 3, 1, 16, 16), (5, 4, 2, 24, 24), (7, 5, 5, 40, 16), (33, 20, 4, 80, 80), (33, 20, 4, 72, 32),
          (19, 32, 8, 128, 128), (300, 8, 2, 128, 64), (17, 6, 3, 192, 192), (9, 4, 1, 256, 256), (13, 3, 2, 248, 8),
          (6, 64, 1, 96, 48), (5000, 2, 1, 64, 64)]


@pytest.mark.parametrize("T,hq,hk,d,rot", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
def test_against_the_definition(T, hq, hk, d, rot, inter):
    _check(T, hq, hk, d, rot, inter=inter)


@pytest.mark.parametrize("T,hq,hk,d,rot", SHAPES + [(11, 21, 4, 48, 48), (40, 9, 3, 160, 80), (3, 33, 2, 88, 88), (70, 13, 13, 72, 72)])
@pytest.mark.parametrize("inter", [False, True])
def test_a_rotation_alone(T, hq, hk, d, rot, inter):
    """Lanes of a head are then no power of two (5 for 80 dims, 9 for 72, 3 for 24 or 48)."""
    _check(T, hq, hk, d, rot, inter=inter, norm=False)


@pytest.mark.parametrize("kw", [dict(norm=False), dict(norm=False, inter=True, axes=3), dict(axes=3), dict(axes=2, wide=True),
                                dict(far=1 << 24), dict(far=(1 << 31) - 5001), dict(far=-(1 << 31), wide=True), dict(factor=1.3),
                                dict(wt=torch.float32, offset=1.0), dict(norm=False, factor=0.5, far=123456)])
@pytest.mark.parametrize("d,rot", [(128, 128), (72, 40)])
def test_forms(kw, d, rot):
    _check(65, 6, 2, d, rot, **kw)


def test_a_norm_alone_and_queries_alone():
    _check(37, 6, 2, 64, 0)
    r, o, (wq, _) = _rope(21, 64, 64)
    q, dq = _bf((21, 6, 64), 1), _bf((21, 6, 64), 2)
    with pytest.raises(M.LmError):
        M.qkrope_fwd(q, None, r)  # (w_k without keys)
    r.w_k = None
    fw, bw = M.qkrope_fwd(q, None, r), M.qkrope_bwd(q, None, dq, None, r)
    assert fw["k"] is None and bw["dk"] is None and bw["dw_k"] is None
    _near("q", fw["q"], O.qkrope_forward(host64(q), w=wq, **o), 2.0 ** -18)
    _near("dq", bw["dq"], O.qkrope_backward(host64(q), host64(dq), w=wq, **o)[0], 2.0 ** -17)


def test_norm_without_weights_and_the_tokens_index():
    q, k = _bf((50, 4, 64), 1), _bf((50, 2, 64), 2)
    f = (1e4 ** (-torch.arange(32).double() / 32)).float().cuda()
    fw = M.qkrope_fwd(q, k, M.QkRope(inv_freq=f, norm=True))
    a = O.qkrope_angles(50, f.cpu().numpy())
    for n, x in (("q", q), ("k", k)):
        _near(n, fw[n], O.qkrope_forward(host64(x), a, norm=True), 2.0 ** -18)


@pytest.mark.parametrize("fr", [1.0, 3.0, 0.0, 1e-30, 2.0 ** -140, 1e6, 2.0 ** 30, -0.5])
def test_frequencies_of_every_size(fr):
    """Also negative and subnormal ones, and whole numbers of radians per position that are many turns."""
    q = _bf((40, 1, 8), 1)
    f = torch.tensor([fr, 0.1, fr, 0.0], device="cuda")
    fw = M.qkrope_fwd(q, None, M.QkRope(inv_freq=f, interleaved=True))
    _near("q", fw["q"], O.qkrope_forward(host64(q), O.qkrope_angles(40, f.cpu().numpy()), True), 2.0 ** -18)


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (5, 5, 72)])
def test_slices_of_one_buffer_and_in_place(hq, hk, d):
    T = 70
    r, _, _ = _rope(T, d, d // 16 * 16)
    qkv = _bf((T, hq + 2 * hk, d), 5)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    want = M.qkrope_fwd(q.contiguous(), k.contiguous(), r)
    got = M.qkrope_fwd(q, k, r)
    assert all(torch.equal(got[n], want[n]) for n in want)
    dbuf = _bf((T, hq + hk, d), 6)
    dq, dk = dbuf[:, :hq], dbuf[:, hq:]
    bw = M.qkrope_bwd(q, k, dq, dk, r)
    keep = v.clone()
    out = torch.full((T, hk + hq, d), 7.0, device="cuda").bfloat16()  # the other way round, in another buffer
    M.qkrope_fwd(q, k, r, q_out=out[:, hk:], k_out=out[:, :hk])
    assert torch.equal(out[:, hk:], want["q"]) and torch.equal(out[:, :hk], want["k"])
    head_major = torch.empty((hq, T, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(M.qkrope_fwd(q, k, r, q_out=head_major)["q"], want["q"])
    bi = M.qkrope_bwd(q, k, dq, dk, r, dq_in=dq, dk_in=dk)
    assert bi["dq"] is dq and all(torch.equal(bi[n], bw[n]) for n in ("dq", "dk", "dw_q", "dw_k"))
    assert torch.equal(dbuf[:, :hq], bw["dq"]) and torch.equal(dbuf[:, hq:], bw["dk"])
    got = M.qkrope_fwd(q, k, r, q_out=q, k_out=k)
    assert torch.equal(qkv[:, :hq], want["q"]) and torch.equal(qkv[:, hq:hq + hk], want["k"]) and torch.equal(v, keep)
    with pytest.raises(M.LmError) as e:
        M.qkrope_fwd(q, k, r, q_out=qkv[:, 1:hq + 1])
    assert e.value.status == L.LM_ERR_ALIAS


def test_the_same_bits_in_a_graph_and_on_a_stream():
    q, k, dq, dk, r, fw, bw = _check(200, 8, 2, 128, 128)
    ws = bw["ws"]

    def step(**kw):
        a, b = M.qkrope_fwd(q, k, r, **kw), M.qkrope_bwd(q, k, dq, dk, r, ws=ws, **kw)
        return [a["q"], a["k"], b["dq"], b["dk"], b["dw_q"], b["dw_k"]]

    want = [fw["q"], fw["k"], bw["dq"], bw["dk"], bw["dw_q"], bw["dw_k"]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_no_tokens():
    r, _, _ = _rope(0, 64, 64)
    q, k = _bf((0, 4, 64), 1), _bf((0, 2, 64), 2)
    fw, bw = M.qkrope_fwd(q, k, r), M.qkrope_bwd(q, k, q, k, r)
    assert fw["q"].shape == q.shape and not bw["dw_q"].any() and not bw["dw_k"].any()


def test_a_row_of_zeros_and_one_that_is_nan():
    r, _, _ = _rope(4, 64, 64)
    q, dq = _bf((4, 2, 64), 1), _bf((4, 2, 64), 2)
    q[1, 0] = 0
    r.w_k = None
    want = M.qkrope_fwd(q, None, r)["q"].clone()
    assert not want[1, 0].any()
    gz = M.qkrope_bwd(q, None, dq, None, r)["dq"].clone()
    assert torch.isfinite(gz).all()
    q[2, 1, 5] = float("nan")
    got, g = M.qkrope_fwd(q, None, r)["q"], M.qkrope_bwd(q, None, dq, None, r)["dq"]
    assert got[2, 1].isnan().all() and g[2, 1].isnan().all()
    keep = torch.ones(4, 2, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(got[keep], want[keep]) and torch.equal(g[keep], gz[keep])


def test_offsets_past_32_bits():
    T, stride = 3, 1 << 31  # tokens 4 GB apart
    big = torch.empty(2 * stride + 4 * 64, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((T, 4, 64), (stride, 64, 1))
    q.copy_(_bf((T, 4, 64), 1))
    r, o, (wq, _) = _rope(T, 64, 64)
    r.w_k = None
    _near("q", M.qkrope_fwd(q, None, r)["q"], O.qkrope_forward(host64(q.contiguous()), w=wq, **o), 2.0 ** -18)
    assert torch.equal(M.qkrope_fwd(q.contiguous(), None, r)["q"], M.qkrope_fwd(q, None, r, q_out=q)["q"])
