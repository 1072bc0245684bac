"""The backward of prompts of few rows and heads, whose walks are cut into
pieces, against the token recurrence in 64 bits: with the bounds of the uncut
walks (gradients in bf16 1e-2; dg and the state's gradient, fp32 from split
products, 1e-4 and 1e-5), and bit for bit against itself."""
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


CASES = [  # B, H, Hk, T, Dk, Dv, lens, per head, token-major, launches
    (1, 1, 1, 3333, 128, 128, None, False, False, 3),
    (2, 2, 1, 2500, 128, 64, None, False, True, 4),
    (1, 2, 2, 6000, 64, 128, [6000], True, False, 6),
    (1, 2, 2, 6000, 128, 128, [1, 0, 5000, 130, 0, 869, 0], False, True, 5),
    (1, 4, 2, 6000, 64, 64, [700, 65, 2, 4800, 433], False, True, 6),
]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("B,H,Hk,T,Dk,Dv,lens,per_head,token_major,launches", CASES)
def test_backward(B, H, Hk, T, Dk, Dv, lens, per_head, token_major, launches, states):
    d = inputs(B, H, Hk, T, Dk, Dv, "bf16", 31 + T, lens, per_head, token_major=token_major)
    s0, dsf = (d["s0"], d["dsf"]) if states else (None, None)
    call = lambda: binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=s0, dfinal_state=dsf,  # noqa: E731
                                             cu_seqlens=None if lens is None else offsets(lens), scale=0.7)
    before = binding.launch_count()
    got = call()
    assert binding.launch_count() == before + launches  # two of walks, the gradients, tables and sums
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], s0, dsf, lens, 0.7)
    for name, x, r in zip(("dq", "dk", "dv"), got, want):
        assert rel_err(x, r) <= TOL_BF16, name
    assert rel_err(got[3], want[3]) <= 1e-4
    if states:
        assert rel_err(got[4], want[4]) <= 1e-5
    for x, y in zip(got, call()):
        assert (x is None and y is None) or torch.equal(x, y)
    assert binding.device_error() == 0


def test_cleared_states():
    """Gates of -inf inside and at the ends of pieces."""
    d = inputs(1, 2, 2, 3000, 128, 128, "bf16", 5)
    d["g"][:, 0, 1000:1010] = -float("inf")
    d["g"][:, 1, ::500] = -1e4
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["s0"], dfinal_state=d["dsf"])
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["s0"], d["dsf"])
    for name, x, r, tol in zip(("dq", "dk", "dv", "dg", "ds0"), got, want, (TOL_BF16,) * 3 + (1e-4, 1e-5)):
        assert rel_err(x, r) <= tol, name


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("T,lens", [(1, None), (3, None), (64, None), (90, [1, 1, 64, 0, 24])])
def test_few_tokens_of_heads_that_cancel(T, lens, Dk, Dv):
    """Two value heads of one key whose gradients nearly cancel in dq and dk: what
    remains is 2^-4 of them, so that a term rounded to bf16 (2^-9) would be 2^-5 off."""
    d = inputs(2 if lens is None else 1, 2, 1, T, Dk, Dv, "bf16", 17, lens)
    d["g"][:, 1] = d["g"][:, 0]
    d["do"][:, 1] = -(d["do"][:, 0].float() * 1.0625).bfloat16()
    d["v"][:, 1] = d["v"][:, 0]
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=None if lens is None else offsets(lens))
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], None, None, lens)
    for name, x, r in zip(("dq", "dk", "dv"), got, want):
        assert rel_err(x, r) <= TOL_BF16, name
