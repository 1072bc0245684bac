"""Outputs of the caller's beside what a call reads, and over it: columns of one buffer
serve as input and output, memory that the call still reads is refused."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_causal_conv import inputs as conv_inputs
from tests.test_gpu_ssm_scan import forward, inputs as scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def beside(t, more):
    """t as the first columns of a wider buffer, and `more` columns behind them."""
    buf = torch.full((*t.shape[:-1], t.shape[-1] + more), 7.0, device="cuda", dtype=t.dtype)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]], buf[..., t.shape[-1]:]


def test_columns_of_one_buffer():
    d = conv_inputs(2, 700, 64, 4, "bf16", 1)
    want = binding.causal_conv_fwd(d["x"], d["w"], d["b"], initial_window=d["win"])[0]
    x, y = beside(d["x"], 64)
    got = binding.causal_conv_fwd(x, d["w"], d["b"], initial_window=d["win"], y=y)[0]
    assert torch.equal(got, want) and torch.equal(x, d["x"])
    s = scan_inputs(2, 700, 64, 16, "f32", 2)
    want = forward(s)
    x, y = beside(s["x"], 64)
    got = forward(dict(s, x=x), y=y)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(x, s["x"])


def test_over_what_is_read():
    d = conv_inputs(2, 3, 64, 4, "bf16", 1)
    refused = lambda: pytest.raises(ValueError, match="share memory")  # noqa: E731
    with refused():
        binding.causal_conv_fwd(d["x"], d["w"], initial_window=d["win"], y=d["win"])
    for w, out in ((d["win"], None), (d["dwin"], d["win"])):
        with refused():
            binding.causal_conv_step(d["x"][:, 0], d["w"], w, window_out=out, y=d["win"].view(6, 64)[2:4])
    s = scan_inputs(2, 16, 64, 16, "f32", 2)
    with refused():
        forward(s, y=s["s0"].view(2, 16, 64))
    row = [s["x"][:, 0], s["dt"][:, 0], s["A"], s["B"][:, 0], s["C"][:, 0]]
    for state, out in ((s["s0"], None), (s["dsf"], s["s0"])):
        with refused():
            binding.ssm_step(*row, state, state_out=out, y=s["s0"].view(32, 64)[3:5])
