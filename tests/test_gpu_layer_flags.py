"""Flags of the layer operators go by their truth, as everywhere in the binding:
1 or numpy's True is True.  Calls with one and the other launch the same kernels
on the same arguments and give equal bits; those without differ."""
import numpy as np
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_linattn import inputs

pytestmark = pytest.mark.gpu

TRUE, FALSE = [1, np.bool_(True), "yes"], [0, np.bool_(False), None, ""]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("given,meant", [(x, True) for x in TRUE] + [(x, False) for x in FALSE])
def test_l2norm(given, meant):
    gen = torch.Generator().manual_seed(1)
    q, k, v = (3 * torch.randn(2, 2, 64, generator=gen).cuda().bfloat16() for _ in range(3))
    g, beta = -torch.rand(2, 2, generator=gen).cuda(), torch.rand(2, 2, generator=gen).cuda().bfloat16()
    start = torch.randn(4, 2, 64, 64, generator=gen).cuda()

    def call(l2norm):
        pool = start.clone()
        return binding.gdn_step(q, k, v, beta, g, pool, l2norm=l2norm), pool

    for x, same, other in zip(call(given), call(meant), call(not meant)):
        assert torch.equal(x, same) and not torch.equal(x, other)


@pytest.mark.parametrize("given,meant", [(x, True) for x in TRUE] + [(x, False) for x in FALSE])
def test_simt(given, meant):
    d = inputs(1, 2, 1, 200, 128, 128, "bf16", 4)
    args = d["q"], d["k"], d["v"], d["g"]
    x, same, other = (binding.linattn_chunk_fwd(*args, simt=s)[0] for s in (given, meant, not meant))
    assert torch.equal(x, same) and not torch.equal(x, other)
    x, same, other = (binding.linattn_chunk_bwd(*args, d["do"], simt=s)[0] for s in (given, meant, not meant))
    assert torch.equal(x, same) and not torch.equal(x, other)


def test_what_has_no_truth():
    """A flag whose truth cannot be told raises what asking for it raises."""
    d = inputs(1, 1, 1, 8, 64, 64, "bf16", 4)
    args = d["q"], d["k"], d["v"], d["g"]
    for name in ("output_final_state", "simt"):
        with pytest.raises(ValueError, match="ambiguous"):
            binding.linattn_chunk_fwd(*args, **{name: np.zeros(2)})
    with pytest.raises(ValueError, match="ambiguous"):
        binding.linattn_chunk_bwd(*args, d["do"], simt=np.zeros(2))
    # no error is left behind
    assert binding.linattn_chunk_fwd(*args)[1] is None
