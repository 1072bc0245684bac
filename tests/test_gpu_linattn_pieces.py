"""Prompts of few rows and heads, whose sequences are cut into pieces that start
from the shares before them: against the token recurrence in 64 bits, with the
bounds of the uncut walk (bf16 outputs 1e-2; final states, fp32 from exact
products, 1e-5), and bit for bit against themselves."""
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


CASES = [  # B, H, Hk, T, Dk, Dv, lens, per head, token-major
    (1, 1, 1, 3333, 128, 128, None, False, False),
    (3, 2, 1, 2500, 128, 128, None, False, True),
    (1, 2, 2, 4000, 64, 128, [4000], True, False),
    (1, 3, 3, 4000, 128, 64, [1, 0, 3500, 130, 0, 369], False, True),
    (1, 4, 2, 4000, 128, 128, [700, 65, 2, 2800, 433], False, True),
    (1, 2, 1, 4000, 64, 64, [1900, 2100], False, False),
]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("B,H,Hk,T,Dk,Dv,lens,per_head,token_major", CASES)
def test_forward(B, H, Hk, T, Dk, Dv, lens, per_head, token_major, states):
    d = inputs(B, H, Hk, T, Dk, Dv, "bf16", 7 + T, lens, per_head, token_major=token_major)
    s0 = d["s0"] if states else None
    call = lambda: binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=s0, output_final_state=states,  # noqa: E731
                                             cu_seqlens=None if lens is None else offsets(lens), scale=0.7)
    launches = binding.launch_count()
    o, sf = call()
    assert binding.launch_count() == launches + 2  # the plan and the walk
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"], s0, lens, 0.7)
    assert rel_err(o, ro) <= TOL_BF16
    if states:
        assert rel_err(sf, rs) <= 1e-5
    for _ in range(3):
        again, sf2 = call()
        assert torch.equal(again, o) and (sf is None or torch.equal(sf, sf2))
    assert binding.device_error() == 0


def test_strong_decays_and_cleared_states():
    """Gates of -inf and far below -100 inside and at the ends of pieces."""
    d = inputs(1, 2, 2, 3000, 128, 128, "bf16", 5)
    d["g"][:, 0, 1000:1010] = -float("inf")
    d["g"][:, 1, ::500] = -1e4
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], output_final_state=True)
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"], d["s0"])
    assert rel_err(o, ro) <= TOL_BF16 and rel_err(sf, rs) <= 1e-5


def test_tokens_of_no_sequence():
    """Offsets that leave tokens out: zeros there, and what lies there (an
    infinity, a NaN) reaches nothing else."""
    lens, first, T = [4200, 0, 37, 130], 21, 4500
    d = inputs(1, 2, 1, T, 128, 128, "bf16", 3, lens)
    end = first + sum(lens)
    for name in ("q", "k", "v"):
        d[name][:, :, :first] = float("nan")
        d[name][:, :, end:] = float("inf")
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], output_final_state=True,
                                      cu_seqlens=offsets(lens, first))
    clean = {n: torch.nan_to_num(d[n].float(), 0.0, 0.0, 0.0) for n in ("q", "k", "v")}
    ro, rs = ref.linattn(clean["q"], clean["k"], clean["v"], d["g"], d["s0"], lens, first=first)
    assert float(o[:, :, :first].abs().max()) == 0.0 and float(o[:, :, end:].abs().max()) == 0.0
    assert rel_err(o, ro) <= TOL_BF16 and rel_err(sf, rs) <= 1e-5


def test_on_another_stream():
    """Two streams at once, each call with its own workspace."""
    d = inputs(1, 2, 2, 4000, 128, 128, "bf16", 9)
    want, _ = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(4):
        for s in streams:
            outs.append(binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and binding.device_error() == 0
