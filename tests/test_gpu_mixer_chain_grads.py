"""The gradients that one operator next to a mixer hands to the one before it, each
against 64 bits at the inputs that its call was given: the block norm's at the h
that its forward stored, then the scan's x, which the convolution's backward takes."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import mixer_reference as ref
from tests.gpu_util import ensure_lib
from tests.test_gpu_causal_conv import close as conv_close
from tests.test_gpu_gated_norm import close as norm_close
from tests.test_gpu_mixer_chain import C, N, weights
from tests.test_gpu_ssm_scan import close as scan_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_gradients_between_the_operators():
    w = weights(11)
    gen = torch.Generator().manual_seed(12)
    x, res, dy, dh = (torch.randn(2, 70, C, generator=gen).bfloat16().cuda() for _ in range(4))
    u, _, h0 = binding.rms_norm_fwd(x, w["pre"], residual=res)
    xz = u @ w["inp"]
    xc, z = xz[..., :C], xz[..., C:]
    xs, _ = binding.causal_conv_fwd(xc, w["taps"], w["bias"])
    dbc = xs @ w["dbc"]
    dt, B, Cm = dbc[..., :C], dbc[..., C:C + N], dbc[..., C + N:]
    y, _ = binding.ssm_scan_fwd(xs, dt, w["A"], B, Cm, D=w["D"], z=z, dt_bias=w["dt_bias"])
    o = y @ w["out"]
    _, h1 = binding.block_norm_fwd(o, h0, w["post"], w["scale"], w["nxt"])

    do, dres, dpost, dscale, dnxt = binding.block_norm_bwd(dy, dh, o, h1, w["post"], w["scale"], w["nxt"])
    flat = lambda t: ref.wide(t).flatten(0, 1)  # noqa: E731
    leaf = ref.leaves(h=h1.flatten(0, 1), w=w["nxt"])
    norm = leaf["h"] / ((leaf["h"] ** 2).mean(-1, keepdim=True) + 1e-6).sqrt() * leaf["w"]
    outer = ref.grads((norm, leaf["h"]), (flat(dy), flat(dh)), leaf)
    leaf = ref.leaves(x=o.flatten(0, 1), w1=w["post"], s=w["scale"])
    _, inner = ref.block(leaf["x"], torch.zeros(140, C, dtype=torch.float64), leaf["w1"], leaf["s"])
    want = ref.grads((inner,), (outer["h"],), leaf)
    many = 1e-5 + 140 ** 0.5 * 2.0 ** -22
    norm_close(dres.flatten(0, 1), outer["h"], "bf16")
    norm_close(do.flatten(0, 1), want["x"], "bf16")
    for got, t in ((dpost, want["w1"]), (dscale, want["s"]), (dnxt, outer["w"])):
        norm_close(got, t, "f32", many)

    dyo = do @ w["out"].t()
    dxs = binding.ssm_scan_bwd(xs, dt, w["A"], B, Cm, dyo, D=w["D"], z=z, dt_bias=w["dt_bias"])[0]
    leaf = ref.leaves(x=xs, dt=dt, A=w["A"], B=B, C=Cm, D=w["D"], z=z, bias=w["dt_bias"])
    scan_close(dxs, ref.grads((ref.scan(*leaf.values())[0],), (ref.wide(dyo),), leaf)["x"], "bf16")
    dxc = binding.causal_conv_bwd(xc, w["taps"], dxs, w["bias"])[0]
    leaf = ref.leaves(x=xc, w=w["taps"], b=w["bias"])
    conv_close(dxc, ref.grads((ref.conv(*leaf.values())[0],), (ref.wide(dxs),), leaf)["x"], "bf16")
