"""The residual RMS norm, its e4m3 output and its backward against 64 bits.
fp32 sums of up to 33,000 squares: 1e-5 relative holds h, y, dx and dw in fp32;
bf16 outputs are a rounding (2^-9) away: 1e-2 with the library's target.  An
e4m3 value is within half a step of y / scale: 2^-4 of itself, or 2^-10 under
the normal range (1e-5 more for the arithmetic)."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, ensure_lib, rel_err

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [(1, 2048), (3, 1), (5, 77), (4, 96), (7, 1000), (2, 2056), (33, 128), (300, 2048), (2, 5120), (1, 8200),
         (2, 16384), (1, 33000)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def inputs(rows, C, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=randn(rows, C), res=3 * randn(rows, C), dy=randn(rows, C))
    d = {n: t.to(DT[dtype]).cuda() for n, t in d.items()}
    d["w"] = (1 + 0.3 * randn(C)).cuda()
    return d


def tol(dtype):
    return TOL_BF16 if dtype == "bf16" else 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("rows,C", SIZES)
def test_norm(rows, C, residual, weight, dtype):
    d = inputs(rows, C, dtype, C)
    res, w = d["res"] if residual else None, d["w"] if weight else None
    y, scales, h = binding.rms_norm_fwd(d["x"], w, residual=res)
    want_h, want_y = ref.rms_norm(d["x"], w, res)
    assert scales is None and y.dtype == DT[dtype]
    assert rel_err(h, want_h) <= tol(dtype) and rel_err(y, want_y) <= tol(dtype)
    if not residual:
        assert h is d["x"]


def check_e4m3(y, scales, want, group):
    rows, C = want.shape
    parts = want.reshape(rows, -1, group or C)
    scales = scales.double().cpu()
    assert scales.shape == parts.shape[:2]
    want_s = (parts.abs().amax(-1) / 448).clamp_min(1e-12)
    assert float(((scales - want_s).abs() / want_s).max()) <= 1e-5
    z = parts / scales[..., None]
    got = y.float().double().cpu().reshape(parts.shape)
    assert bool(((got - z).abs() <= torch.maximum(z.abs() * (2 ** -4 + 1e-5), torch.tensor(2.0 ** -10 + 1e-5))).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C,group", [(3, 2048, 128), (5, 96, 32), (4, 192, 64), (2, 5120, 128), (6, 1000, 0),
                                          (3, 77, 0), (1, 1, 0), (2, 2048, 0), (1, 16384, 128), (1, 33000, 0)])
def test_e4m3(rows, C, group, dtype):
    d = inputs(rows, C, dtype, rows)
    y, scales, h = binding.rms_norm_fwd(d["x"], d["w"], residual=d["res"], out_dtype=torch.float8_e4m3fn, group=group)
    want_h, want_y = ref.rms_norm(d["x"], d["w"], d["res"])
    assert y.dtype == torch.float8_e4m3fn and rel_err(h, want_h) <= tol(dtype)
    check_e4m3(y, scales, want_y, group)


def test_rows_of_zeros_and_bad_rows():
    """A row of zeros gives zeros and the smallest scale; a NaN or an infinity
    stays in its row and shows in its scale."""
    d = inputs(4, 256, "bf16", 1)
    d["x"][0] = 0
    d["x"][2, 5] = float("nan")
    d["x"][3, 7] = float("inf")
    y, scales, _ = binding.rms_norm_fwd(d["x"], d["w"], out_dtype=torch.float8_e4m3fn, group=128)
    assert float(y[0].float().abs().max()) == 0.0 and float(scales[0].max()) == pytest.approx(1e-12)
    _, want = ref.rms_norm(d["x"][1:2], d["w"])
    check_e4m3(y[1:2], scales[1:2], want, 128)
    assert bool(scales[2].isnan().all())
    assert bool(scales[3, 0].isnan())  # inf * 0
    z, _, _ = binding.rms_norm_fwd(d["x"], d["w"])
    assert bool(z[2].isnan().all()) and bool(z[:2].isfinite().all())


def test_shapes_empty_and_stream():
    d = inputs(12, 64, "bf16", 1)
    x = d["x"].reshape(3, 4, 64)
    y, scales, _ = binding.rms_norm_fwd(x, d["w"], out_dtype=torch.float8_e4m3fn, group=32)
    assert y.shape == (3, 4, 64) and scales.shape == (3, 4, 2)
    y, _, _ = binding.rms_norm_fwd(x[:0], d["w"])
    assert y.shape == (0, 4, 64)
    dx, dw = binding.rms_norm_bwd(x[:0], x[:0], d["w"])
    assert dx.shape == (0, 4, 64) and float(dw.abs().max()) == 0.0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _, _ = binding.rms_norm_fwd(d["x"], d["w"], stream=s)
    s.synchronize()
    assert rel_err(y, ref.rms_norm(d["x"], d["w"])[1]) <= TOL_BF16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, False)])
@pytest.mark.parametrize("rows,C", SIZES + [(1500, 256)])
def test_backward(rows, C, residual, weight, dtype):
    d = inputs(rows, C, dtype, C + 1)
    res, w = d["res"] if residual else None, d["w"] if weight else None
    dx, dw = binding.rms_norm_bwd(d["dy"], d["x"], w, dresidual=res)
    want_dx, want_dw = ref.rms_norm_bwd(d["dy"], d["x"], w, res)
    # C = 1: dx of the norm alone is eps-small against its two terms; measured against them
    floor = float((d["dy"].double() / d["x"].double().abs().clamp_min(1e-3)).abs().max()) if C == 1 else 0.0
    err = float((dx.double().cpu() - want_dx).abs().max()) / max(float(want_dx.abs().max()), floor)
    assert err <= tol(dtype)
    assert rel_err(dw, want_dw) <= 1e-5
    again = binding.rms_norm_bwd(d["dy"], d["x"], w, dresidual=res)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_against_differences():
    d = inputs(4, 64, "f32", 9)
    dx, dw = binding.rms_norm_bwd(d["dy"], d["x"], d["w"])
    gen = torch.Generator().manual_seed(2)
    x, w, dy = (d[n].double().cpu() for n in ("x", "w", "dy"))
    loss = lambda x, w: float((ref.rms_norm(x, w)[1] * dy).sum())  # noqa: E731
    for base, grad, f in ((x, dx, lambda z: loss(z, w)), (w, dw, lambda z: loss(x, z))):
        u = torch.randn(base.shape, generator=gen, dtype=torch.float64)
        want = (f(base + 1e-6 * u) - f(base - 1e-6 * u)) / 2e-6
        terms = grad.double().cpu() * u
        assert abs(float(terms.sum()) - want) <= 1e-4 * float(terms.square().sum().sqrt())


def test_refusals():
    d = inputs(4, 256, "bf16", 1)
    f = binding.rms_norm_fwd
    with pytest.raises(TypeError):
        f(d["x"].half(), d["w"])
    with pytest.raises(TypeError):
        f(d["x"], d["w"].bfloat16())
    with pytest.raises(ValueError):
        f(d["x"], d["w"][:100])
    with pytest.raises(ValueError):
        f(d["x"].t(), d["w"])
    with pytest.raises(TypeError):
        f(d["x"], d["w"], residual=d["res"].float())
    with pytest.raises(TypeError):
        f(d["x"], d["w"], out_dtype=torch.float16)
    for group in (48, 256):
        with pytest.raises(ValueError):
            f(d["x"], d["w"], out_dtype=torch.float8_e4m3fn, group=group)
    with pytest.raises(ValueError):
        f(d["x"], d["w"], group=128)
    with pytest.raises(binding.GdnError):
        f(d["x"], d["w"], eps=-1.0)
    with pytest.raises(ValueError):
        binding.rms_norm_bwd(d["dy"][:2], d["x"], d["w"])
    with pytest.raises(binding.GdnError):
        binding.rms_norm_bwd(d["dy"], d["x"], d["w"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
