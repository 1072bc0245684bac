"""The example of a state space layer runs, and its gradients are those of its loss: each
weight's against differences of the same layer in 64 bits."""
import pytest
import torch

from examples.state_space_layer import Layer, main
from gated_delta_rule_47_gb300 import binding
from tests import mixer_reference as ref
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_example_runs(capsys):
    main()
    out = capsys.readouterr().out
    assert "served" in out and "trained" in out and binding.device_error() == 0


def test_gradients():
    """bf16 activations between the operators, each rounded to 2^-8 of itself: about ten of them in a row (2^-5 at
    most) between a gradient and the difference of the loss without any rounding; gradients are compared along
    themselves, where nothing cancels."""
    layer = Layer(C=64, Di=64, N=8, W=4, seed=3)
    gen = torch.Generator().manual_seed(4)
    x, res = (torch.randn(1, 40, 64, generator=gen).bfloat16().cuda() for _ in range(2))
    target = torch.randn(1, 40, 64, generator=gen).cuda()
    _, g = layer.train_step(x, res, target)
    w = {n: ref.wide(getattr(layer, n)) for n in ("win", "wdbc", "wout", "taps", "bias", "A", "D", "dt_bias", "pre", "post", "scale", "next")}
    w["x"] = ref.wide(x)

    def loss(w):
        norm = lambda u, s: u / ((u * u).mean(-1, keepdim=True) + 1e-6).sqrt() * s  # noqa: E731
        h0 = w["x"] + ref.wide(res)
        xz = norm(h0, w["pre"]) @ w["win"]
        xs, _ = ref.conv(xz[..., :64], w["taps"], w["bias"])
        dt, B, C = (xs @ w["wdbc"]).split([64, 8, 8], -1)
        y, _ = ref.scan(xs, dt, w["A"], B, C, w["D"], xz[..., 64:], w["dt_bias"])
        h = h0 + w["scale"] * norm(y @ w["wout"], w["post"])
        return float((norm(h, w["next"]) - ref.wide(target)).square().mean())
    for n, t in w.items():
        along = ref.wide(g[n])
        unit = along / along.norm()
        step = 1e-5 * max(1.0, float(t.norm()))
        slope = (loss({**w, n: t + step * unit}) - loss({**w, n: t - step * unit})) / (2 * step)
        assert abs(slope - float(along.norm())) <= 2.0 ** -5 * abs(slope), n
