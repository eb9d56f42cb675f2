"""A caller's buffer for a result that a call does not have (addnorm_fwd, addnorm_bwd) is not returned as one."""
import pytest
import torch

from bwd_lora_mlp_gb300 import build as B
from bwd_lora_mlp_gb300 import layer as M
from bwd_lora_mlp_gb300 import lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    L.load()


def test_results_that_are_not_there():
    h, y, spare = (torch.full((5, 64), c, dtype=torch.bfloat16, device="cuda") for c in (1.0, 2.0, 7.0))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    fw = M.addnorm_fwd(h, y, M.AddNorm(), x=spare)
    assert fw["x"] is None and torch.all(fw["h"] == 3)
    n = M.AddNorm(w_in=w)
    fw = M.addnorm_fwd(h, None, n, h_out=spare)
    assert fw["h"] is h
    assert M.addnorm_bwd(h, None, None, h, fw, n, dy=spare)["dy"] is None
    assert torch.all(spare == 7)
    with pytest.raises(ValueError):  # (a buffer that would not do is still refused)
        M.addnorm_fwd(h, y, M.AddNorm(), x=spare[:, :32])
