"""Backward of the selective state space scan behind a sequence whose last state is not
finite: the tokens of no sequence behind it, and the room behind a row's last token,
get and give nothing.  By the definition an infinite x in the last token reaches the
step's and skip's gradients of its channel and the gradients of that token alone: no
decay works on the state that it makes."""
import pytest
import torch

from tests.gpu_util import ensure_lib
from tests.test_gpu_ssm_scan import backward, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def check(d, cu, last, bad, channel=3):
    """`last`: the token whose x is bad; gradients beside it are those of a finite x there."""
    clean = (forward(d, cu), backward(d, cu))
    d = dict(d, x=d["x"].clone())
    d["x"][0, last, channel] = bad
    y, state = forward(d, cu)
    got = backward(d, cu)
    other = torch.arange(d["x"].shape[2], device="cuda") != channel
    before = torch.arange(d["x"].shape[1], device="cuda") != last
    assert torch.equal(y[:, before], clean[0][0][:, before]) and torch.equal(state[..., other, :], clean[0][1][..., other, :])
    want = clean[1]
    assert torch.equal(got["A"], want["A"]) and torch.equal(got["s0"], want["s0"])
    for n in ("D", "bias"):
        assert torch.equal(got[n][other], want[n][other]), n
    for n in ("x", "dt", "B", "C", "z"):
        assert torch.equal(got[n][:, before], want[n][:, before]), n
    assert torch.equal(got["x"][0, last], want["x"][0, last])  # dx does not depend on x
    for n in ("dt", "z"):
        assert torch.equal(got[n][0, last, other], want[n][0, last, other]), n
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("end", [9, 12, 13, 16, 23])
def test_padding_behind_a_state_that_is_not_finite(end, bad, N, dtype):
    """Padding in the end's own four tokens, in the next four, and in whole blocks behind it."""
    d = inputs(1, 90, 40, N, dtype, end, n_seq=2)
    got = check(d, torch.tensor([2, 5, end], dtype=torch.int32, device="cuda"), end - 1, bad)
    for n in ("x", "dt", "B", "C", "z"):
        assert float(got[n][0, end:].float().abs().max()) == 0.0 and float(got[n][0, :2].float().abs().max()) == 0.0, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 13, 16, 131])
def test_last_token_of_a_row(T, dtype):
    check(inputs(1, T, 40, 16, dtype, T), None, T - 1, float("inf"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_last_token_before_another_sequence(dtype):
    d = inputs(1, 90, 40, 16, dtype, 7, n_seq=3)
    check(d, torch.tensor([0, 21, 21, 90], dtype=torch.int32, device="cuda"), 20, float("inf"))
