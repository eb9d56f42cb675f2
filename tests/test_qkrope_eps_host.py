"""The smallest eps of qkrope's norm (no GPU needed): subnormals are refused, the smallest normal number is not."""
import pytest

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import lib as L

from test_qkrope_abi_host import _args, _bwd, _fwd


@pytest.fixture(scope="module", autouse=True)
def so():
    B.build()
    return L.load()


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_eps(call):
    base = _args()
    with_eps = lambda eps, **kw: dict(base, r=dict(base["r"], eps=eps), **kw)  # noqa: E731
    for eps in (2.0 ** -149, 1e-39, 2.0 ** -127, -1e-6, float("nan")):
        assert call(with_eps(eps)) == L.LM_ERR_SHAPE, eps
    # (no tokens: a call that passes its checks does nothing but clear the sums, and those are not asked for)
    for eps in (2.0 ** -126, 1e-30):
        assert call(with_eps(eps, T=0, dw_q=None, dw_k=None)) == L.LM_OK, eps
