"""gdn_step is the delta rule: without beta it is refused, and nothing is written."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [{}, dict(o=True), dict(l2norm=True)])
def test_no_beta(more):
    ensure_lib()
    q, k, v = (torch.randn(2, 2, 64, device="cuda") for _ in range(3))
    g, pool = -torch.rand(2, 2, device="cuda"), torch.randn(3, 2, 64, 64, device="cuda")
    before = pool.clone()
    if more.get("o"):
        more = dict(o=torch.empty_like(v))
    with pytest.raises(TypeError, match="beta"):
        binding.gdn_step(q, k, v, None, g, pool, **more)
    assert torch.equal(pool, before)
