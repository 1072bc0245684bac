"""The backward of a packed sequence does not depend on what it is packed with:
neither its bits nor the precision that short sequences get."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, ensure_lib, rel_err
from tests.test_gpu_linattn import inputs, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def cancelling(lens, Dk, Dv, seed=17):
    """Two value heads of one key whose gradients cancel in dq and dk to 2^-4: a term
    rounded to bf16 (2^-9) is up to 2^-9 * 2.06 / 0.0625 = 6e-2 of what remains."""
    d = inputs(1, 2, 1, sum(lens), Dk, Dv, "bf16", seed, lens)
    d["g"][:, 1] = d["g"][:, 0]
    d["do"][:, 1] = -(d["do"][:, 0].float() * 1.0625).bfloat16()
    d["v"][:, 1] = d["v"][:, 0]
    return d


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[1, 128], [1, 2, 700], [300, 64, 0, 5, 400], [3, 1500]])
def test_short_sequences_beside_long_ones(lens, Dk, Dv):
    """Each sequence of up to 64 tokens against its own largest gradient: in two
    bf16 terms what is left is the output's own rounding (2^-9, within 1e-2)."""
    d = cancelling(lens, Dk, Dv)
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=offsets(lens))
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, None, lens)
    t = 0
    for n in lens:
        for name, x, r in zip(("dq", "dk", "dv"), got, want):
            if 0 < n <= 64:
                assert rel_err(x[:, :, t:t + n], r[:, :, t:t + n]) <= TOL_BF16, (name, n)
        t += n


@pytest.mark.parametrize("n", [1, 40, 64, 65, 150, 200])
@pytest.mark.parametrize("other", [[700], [1] * 30, [0] * 20 + [300]])
def test_alone_and_packed(n, other):
    lens = [n, *other]
    d = cancelling(lens, 128, 128)
    packed = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=offsets(lens))
    cut = {x: d[x][:, :, :n].contiguous() for x in ("q", "k", "v", "g", "do")}
    alone = binding.linattn_chunk_bwd(*cut.values(), cu_seqlens=offsets([n]))
    row = binding.linattn_chunk_bwd(*cut.values())
    for x, y, z in zip(packed[:4], alone, row):
        assert torch.equal(x[:, :, :n], y) and torch.equal(y, z)
