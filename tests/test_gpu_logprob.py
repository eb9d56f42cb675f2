"""Log probabilities, entropy and top alternatives (logprob_fwd, logprob_bwd) against the fp64 definition.

Tolerances.  Sums run in fp32 over at most 2e5 terms in blocks, exponentials and logarithms within a
few ulp of values of size at most about 30: 1e-5 absolute for logp, lse, entropy and the alternatives.
dlogits: fp32 within 1e-5 of the row's largest value; bf16 one rounding more (2^-8 of the element).
Indices are exact: ties go to the lowest."""
import numpy as np
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L
from oracle import layer as O

from gpu_util import check, host64

pytestmark = pytest.mark.gpu

ABS = 1e-5
BF16_REL = 2.0 ** -8 + 1e-5
F32_REL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def _case(T, V, dtype, seed=0, std=3.0, pad=0, skip=0):
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(T, V + pad + skip, generator=g) * std).to(dtype).cuda()
    x = buf[:, skip:skip + V]
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < 0.2] = -100
    return x, t.cuda(), torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda()


def _near(name, got, want, tol=ABS):
    got, want = host64(got), np.asarray(want)
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), name
    err = np.abs(got[fin] - want[fin]).max(initial=0.0)
    assert err <= tol, (name, err)


def _check(x, t, gl, ge, k, scale, in_place=False):
    f, tn = host64(x), t.cpu().numpy()
    fw = M.logprob_fwd(x, t, k, scale)
    rf = O.logprob_forward(f, tn, k, scale)
    for n in ("logp", "entropy", "lse"):
        _near(n, fw[n], rf[n])
    if k:
        assert np.array_equal(fw["top_ids"].cpu().numpy(), rf["top_ids"])
        _near("top_logp", fw["top_logp"], rf["top_logp"])
    out = x if in_place else None
    d = M.logprob_bwd(x, t, fw, gl, ge, scale, dlogits=out)["dlogits"]
    rd = O.logprob_backward(f, tn, None if gl is None else host64(gl), None if ge is None else host64(ge), scale)
    check("dlogits", host64(d), rd, BF16_REL if x.dtype == torch.bfloat16 else F32_REL)
    return fw


SHAPES = [(1, 1, 0, 0), (3, 7, 0, 0), (5, 255, 1, 0), (64, 1000, 0, 3), (2, 50257, 0, 0), (9, 4099, 5, 1), (40, 32000, 0, 0),
          (1, 131072, 0, 0), (700, 513, 0, 0), (3, 160001, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pad,skip", SHAPES)
def test_against_the_definition(T, V, pad, skip, dtype):
    for k, scale in ((0, 1.0), (min(V, 1), 0.7), (min(V, 32), 1.4)):
        _check(*_case(T, V, dtype, T + V + k, pad=pad, skip=skip), k, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_gradient_at_a_time(dtype):
    x, t, gl, ge = _case(20, 3001, dtype, 4)
    _check(x, t, gl, None, 0, 1.0)
    _check(x, t, None, ge, 0, 1.0)
    _check(x, t.int(), gl, ge, 3, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,pad", [(4096, 0), (5003, 2)])
def test_gradient_in_place_of_the_logits(dtype, V, pad):
    x, t, gl, ge = _case(12, V, dtype, 6, pad=pad)
    _check(x, t, gl, ge, 2, 1.2, in_place=True)


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "few values"])
@pytest.mark.parametrize("V", [33, 5000, 131072])
def test_alternatives_in_hard_orders(order, V):
    """Rows sorted against the scan, all alike, or full of ties."""
    g = torch.Generator().manual_seed(1)
    for dtype in (torch.bfloat16, torch.float32):
        base = {"rising": torch.linspace(-20, 20, V), "falling": torch.linspace(20, -20, V), "equal": torch.full((V,), 1.5),
                "few values": torch.randint(-3, 4, (V,), generator=g).float()}[order]
        x = torch.stack([base, base.roll(V // 3), -base]).to(dtype).cuda()
        t = torch.tensor([0, V - 1, V // 2], device="cuda")
        _check(x, t, torch.ones(3, device="cuda"), torch.ones(3, device="cuda"), 32, 1.0)


def test_infinite_and_missing_logits():
    x, t, gl, ge = _case(6, 5000, torch.float32, 8)
    inf = float("inf")
    x[0, ::2] = -inf                       # half of the vocabulary masked
    t[0] = 2                               # a masked target
    x[1, :] = -inf                         # nothing left
    t[1] = 3
    x[2, :] = -inf
    x[2, 77] = 1.0                         # one left
    t[2] = 77
    x[3, 4999] = torch.finfo(torch.float32).min
    x[4, 0] = -0.0
    fw = M.logprob_fwd(x, t, 5)
    rf = O.logprob_forward(host64(x), t.cpu().numpy(), 5)
    for n in ("logp", "entropy", "lse", "top_logp"):
        _near(n, fw[n], rf[n])
    assert np.array_equal(fw["top_ids"].cpu().numpy(), rf["top_ids"])
    d = M.logprob_bwd(x, t, fw, gl, ge)["dlogits"]
    ref = O.logprob_backward(host64(x), t.cpu().numpy(), host64(gl), host64(ge))
    assert torch.all(d[1] == 0)
    check("dlogits", host64(d), ref, F32_REL)
    bf = x.bfloat16()
    assert torch.all(M.logprob_bwd(bf, t, M.logprob_fwd(bf, t), gl, ge)["dlogits"][1] == 0)


def test_a_nan_stays_in_its_row():
    x, t, gl, ge = _case(4, 3000, torch.float32, 9)
    x[1, 2990] = float("nan")
    fw = M.logprob_fwd(x, t, 3)
    rf = O.logprob_forward(host64(x), t.cpu().numpy(), 3)
    assert np.array_equal(fw["top_ids"].cpu().numpy(), rf["top_ids"])
    assert torch.isnan(fw["lse"][1])
    keep = [0, 2, 3]
    for n in ("logp", "entropy", "lse"):
        _near(n, fw[n][keep], rf[n][keep])


def test_no_tokens_and_outside_targets():
    x = torch.empty((0, 100), dtype=torch.bfloat16, device="cuda")
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    fw = M.logprob_fwd(x, t, 2)
    assert fw["top_ids"].shape == (0, 2) and M.logprob_bwd(x, t, fw)["dlogits"].shape == (0, 100)
    x, t, gl, ge = _case(5, 100, torch.float32, 2)
    t[:] = torch.tensor([-1, 100, 2 ** 40, -2 ** 40, 99], device="cuda")
    fw = _check(x, t, gl, ge, 0, 1.0)
    assert torch.all(fw["logp"][:4] == 0) and fw["logp"][4] < 0


def test_same_bits_again_and_on_a_side_stream():
    x, t, gl, ge = _case(33, 50257, torch.bfloat16, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for stream in (None, None, side):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            fw = M.logprob_fwd(x, t, 20, stream=stream)
            fw["d"] = M.logprob_bwd(x, t, fw, gl, ge, stream=stream)["dlogits"]
        torch.cuda.synchronize()
        runs.append(fw)
    for r in runs[1:]:
        for n in r:
            assert torch.equal(r[n], runs[0][n]), n


def test_gradients_against_differences():
    x, t, gl, ge = _case(8, 400, torch.float32, 12)
    fw = M.logprob_fwd(x, t, scale=0.9)
    d = M.logprob_bwd(x, t, fw, gl, ge, 0.9)["dlogits"]
    step = torch.sign(d) * 0.01

    def f(x):
        o = M.logprob_fwd(x, t, scale=0.9)
        return ((o["logp"].double() * gl).sum() + (o["entropy"].double() * ge).sum()).item()

    said = 2 * (d.double() * step.double()).sum().item()
    assert abs(f(x + step) - f(x - step) - said) <= 1e-3 * abs(said)


def test_offsets_past_32_bits():
    """18000 rows of 131072 bf16 logits: 2.36e9 elements; rows from both ends against the definition."""
    T, V = 18000, 131072
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, V, generator=g, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    gl = torch.randn(T, generator=g, device="cuda")
    fw = M.logprob_fwd(x, t, 4)
    rows = torch.tensor([0, T // 2, T - 2, T - 1], device="cuda")
    f, tn = host64(x[rows]), t[rows].cpu().numpy()
    rf = O.logprob_forward(f, tn, 4)
    for n in ("logp", "entropy", "lse", "top_logp"):
        _near(n, fw[n][rows], rf[n])
    assert np.array_equal(fw["top_ids"][rows].cpu().numpy(), rf["top_ids"])
    d = M.logprob_bwd(x, t, fw, gl)["dlogits"]
    check("dlogits", host64(d[rows]), O.logprob_backward(f, tn, host64(gl[rows])), BF16_REL)
    del x, d
    torch.cuda.empty_cache()


@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_masks_of_the_types_lowest_value_and_huge_logits(scale):
    """bf16 rows whose masked logits are the type's lowest value or -inf, both, nothing else, or lie next to
    huge ones; the entropy is of what is left."""
    low, inf = torch.finfo(torch.bfloat16).min, float("inf")
    x, t, _, _ = _case(7, 3001, torch.bfloat16, 21)
    x[0, ::2], x[0, 1::2] = -inf, low      # the lowest value is what is left
    t[0] = 5
    x[1, ::3] = low
    t[1] = 1
    x[2, :], x[2, 2000] = low, 3e38
    t[2] = 2000
    x[3, :], x[3, 10:20] = -2e36, 2e36
    t[3] = 12
    x[4, :], x[4, 7:9] = -inf, 1e37
    t[4] = 8
    x[5, :] = low
    t[5] = 0
    x[6, ::2], x[6, 1::4] = -inf, low
    t[6] = 3
    fw = M.logprob_fwd(x, t, 1, scale)
    rf = O.logprob_forward(host64(x), t.cpu().numpy(), 1, scale)
    for n in ("logp", "entropy", "top_logp"):
        _near(n, fw[n], rf[n])
    assert np.array_equal(fw["top_ids"].cpu().numpy(), rf["top_ids"])
    lse, want = host64(fw["lse"]), rf["lse"]
    assert np.all(np.abs(lse - want) <= np.maximum(ABS, 2.0 ** -23 * np.abs(want)))  # (one rounding to fp32)
    d = M.logprob_bwd(x, t, fw, torch.ones(7, device="cuda"), None, scale)["dlogits"]
    # (rows 0, 3, 4, 5: lse cannot hold the logarithm of how many equal logits there are beside 1e36 of them)
    assert torch.isfinite(d).all() and torch.all(d[[1, 2, 6]].sum(1).abs() < 0.1)
