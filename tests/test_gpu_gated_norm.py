"""The gated norm by head and the norms around a block against 64 bits.  A value is
rounded once, from fp32: half a step of its type (bf16 2^-8, fp32 2^-24) after fp32
sums of up to 8192 squares and products, each off by at most 13 levels of 2^-24 of
their terms: 1e-5 of the largest value.  Sums over n rows add n^0.5 2^-22."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import mixer_reference as ref
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def close(got, want, dtype, slack=1e-5):
    got = got.double().cpu()
    assert got.shape == want.shape and bool(got.isfinite().all())
    err = (got - want).abs() - HALF[dtype] * want.abs()
    assert float(err.max() if err.numel() else 0) <= slack * max(float(want.abs().max() if want.numel() else 0), 1e-30)


def heads(B, T, H, D, dtype, seed, shared, heads_first=False):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = randn(B, H, T, D).transpose(1, 2) if heads_first else randn(B, T, H, D)
    d = {n: t.to(DT[dtype]).cuda() for n, t in dict(x=x, g=randn(B, T, H, D), dy=randn(B, T, H, D)).items()}
    assert d["x"].stride() == x.stride()
    d["w"] = None if shared is None else (1 + 0.3 * (randn(D) if shared else randn(H, D))).cuda()
    return d


def check_gated(d, dtype, **kw):
    leaf = ref.leaves(x=d["x"], g=d["g"], w=d["w"])
    named = dict(first=kw.get("gate_first", False), sigmoid=kw.get("sigmoid", False))
    want = ref.gated(leaf["x"], leaf["g"], leaf["w"], **named)
    y = binding.gated_norm_fwd(d["x"], d["g"], d["w"], **kw)
    assert y.is_contiguous()
    close(y, want.detach(), dtype)
    grads = ref.grads((want,), (ref.wide(d["dy"]),), leaf)
    dx, dg, dw = binding.gated_norm_bwd(d["dy"], d["x"], d["g"], d["w"], **kw)
    assert dx.stride() == d["x"].stride()
    # x's and the gate's gradients cancel between two terms of up to 1 / sqrt(eps) of dy
    close(dx, grads["x"], dtype)
    close(dg, grads["g"], dtype)
    if d["w"] is not None:
        close(dw, grads["w"], "f32", 1e-5 + d["x"][..., 0].numel() ** 0.5 * 2.0 ** -22)
    again = binding.gated_norm_bwd(d["dy"], d["x"], d["g"], d["w"], **kw)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, dw), again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate_first,sigmoid", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("shared", [True, False])
def test_gated_options(shared, gate_first, sigmoid, dtype):
    check_gated(heads(2, 9, 3, 64, dtype, 1, shared, True), dtype, gate_first=gate_first, sigmoid=sigmoid)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared,heads_first", [(True, False), (False, True), (None, False)])
@pytest.mark.parametrize("B,T,H,D", [(1, 1, 1, 8), (1, 1, 16, 128), (2, 3, 5, 24), (1, 40, 7, 128), (3, 1, 2, 72), (1, 5, 2, 1000),
                                     (1, 3, 1, 2048), (2, 2, 1, 4104), (1, 2, 3, 8192), (1, 700, 32, 64)])
def test_gated(B, T, H, D, shared, heads_first, dtype):
    check_gated(heads(B, T, H, D, dtype, T + D, shared, heads_first), dtype)


def test_gated_slices():
    d = heads(2, 5, 4, 32, "bf16", 3, True)
    wide = torch.randn(2, 5, 4 * 32 * 2 + 16, device="cuda").bfloat16()
    g = wide[..., 16:144].unflatten(-1, (4, 32))
    x = wide[..., 144:].unflatten(-1, (4, 32))
    g.copy_(d["g"]), x.copy_(d["x"])
    assert torch.equal(binding.gated_norm_fwd(x, g, d["w"]), binding.gated_norm_fwd(d["x"], d["g"], d["w"]))
    a, b = binding.gated_norm_bwd(d["dy"], x, g, d["w"]), binding.gated_norm_bwd(d["dy"], d["x"], d["g"], d["w"])
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # one row for all tokens: its gradient is one of every token's
    e = d["x"][:1, :1].expand(2, 5, 4, 32)
    dx = binding.gated_norm_bwd(d["dy"], e, d["g"], d["w"])[0]
    assert torch.equal(dx, binding.gated_norm_bwd(d["dy"], e.contiguous(), d["g"], d["w"])[0])


def test_gated_rows_of_zeros_and_bad_rows():
    d = heads(1, 4, 2, 64, "bf16", 1, True)
    clean = binding.gated_norm_fwd(d["x"], d["g"], d["w"])
    d["x"][0, 0] = 0
    d["x"][0, 1, 1, 5] = float("nan")
    d["g"][0, 2, 0, 7] = float("inf")
    y = binding.gated_norm_fwd(d["x"], d["g"], d["w"])
    assert float(y[0, 0].float().abs().max()) == 0.0 and bool(y[0, 1, 1].isnan().all())
    assert torch.equal(y[0, 1, 0], clean[0, 1, 0]) and torch.equal(y[0, 3], clean[0, 3]) and torch.equal(y[0, 2, 1], clean[0, 2, 1])
    assert int(y[0, 2, 0].isfinite().logical_not().sum()) == 1


def rows(n, C, dtype, seed, groups, weights=True):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {k: t.to(DT[dtype]).cuda() for k, t in dict(x=randn(n, C), res=3 * randn(n, C), dy=randn(n, C), dh=randn(n, C)).items()}
    d["w1"], d["w2"] = ((1 + 0.3 * randn(C)).cuda() if weights else None for _ in range(2))
    d["s"] = (0.5 + 0.1 * randn(*([C] if groups == 1 else [groups, C]))).cuda() if groups else None
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C,groups,weights", [(1, 8, 0, True), (3, 24, 1, True), (8, 2048, 1, False), (12, 256, 4, True),
                                                (7, 1000, 7, True), (2, 4104, 0, False), (3, 8192, 1, True), (900, 64, 3, True),
                                                (700, 128, 1, True), (256, 40, 64, True)])
def test_block(n, C, groups, weights, dtype):
    d = rows(n, C, dtype, n + C, groups, weights)
    y, h = binding.block_norm_fwd(d["x"], d["res"], d["w1"], d["s"], d["w2"])
    wy, wh = ref.block(*(ref.wide(d[k]) for k in ("x", "res", "w1", "s", "w2")))
    close(h, wh, dtype)
    close(y, wy, dtype)
    # the backward at the h that is stored: its norm's share and the residual's, then the first norm's
    leaf = ref.leaves(x=d["x"], h=h, w1=d["w1"], s=d["s"], w2=d["w2"])
    norm = lambda u, w: u / ((u * u).mean(-1, keepdim=True) + 1e-6).sqrt() * (1 if w is None else w)  # noqa: E731
    dres = ref.grads((norm(leaf["h"], leaf["w2"]), leaf["h"]), (ref.wide(d["dy"]), ref.wide(d["dh"])), dict(h=leaf["h"], w2=leaf["w2"]))
    zero = torch.zeros(n, C, dtype=torch.float64)
    _, inner = ref.block(leaf["x"], zero, leaf["w1"], leaf["s"])
    first = ref.grads((inner,), (dres["h"],), dict(x=leaf["x"], w1=leaf["w1"], s=leaf["s"]))
    got = binding.block_norm_bwd(d["dy"], d["dh"], d["x"], h, d["w1"], d["s"], d["w2"])
    close(got[0], first["x"], dtype)
    close(got[1], dres["h"], dtype)
    many = 1e-5 + n ** 0.5 * 2.0 ** -22
    for t, want in zip(got[2:], (first["w1"], first["s"], dres["w2"])):
        if want is None:
            assert t is None
        else:
            close(t, want, "f32", many)
    again = binding.block_norm_bwd(d["dy"], d["dh"], d["x"], h, d["w1"], d["s"], d["w2"])
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    none = binding.block_norm_bwd(d["dy"], None, d["x"], h, d["w1"], d["s"], d["w2"])
    zeros = binding.block_norm_bwd(d["dy"], torch.zeros_like(h), d["x"], h, d["w1"], d["s"], d["w2"])
    assert all(a is b or torch.equal(a, b) for a, b in zip(none, zeros))


def test_differences():
    d = heads(1, 3, 2, 8, "f32", 2, False)
    gen = torch.Generator().manual_seed(2)
    for kw in (dict(), dict(gate_first=True), dict(sigmoid=True)):
        named = dict(first=kw.get("gate_first", False), sigmoid=kw.get("sigmoid", False))
        got = dict(zip("xgw", binding.gated_norm_bwd(d["dy"], d["x"], d["g"], d["w"], **kw)))
        base = {n: ref.wide(d[n]) for n in "xgw"}
        for n in "xgw":
            u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
            f = lambda e: float((ref.gated(**{**base, n: base[n] + e * u}, **named) * ref.wide(d["dy"])).sum())  # noqa: E731, B023
            terms = got[n].double().cpu() * u
            assert abs(float(terms.sum()) - (f(1e-6) - f(-1e-6)) / 2e-6) <= 1e-4 * float(terms.square().sum().sqrt())


def test_shapes_empty_and_stream():
    d = rows(12, 64, "bf16", 1, 3)
    x, res = d["x"].reshape(3, 4, 64), d["res"].reshape(3, 4, 64)
    y, h = binding.block_norm_fwd(x, res, d["w1"], d["s"], d["w2"])
    want = binding.block_norm_fwd(d["x"], d["res"], d["w1"], d["s"], d["w2"])
    assert torch.equal(y.flatten(0, 1), want[0]) and torch.equal(h.flatten(0, 1), want[1])
    y, h = binding.block_norm_fwd(x[:0], res[:0], d["w1"], None, d["w2"])
    assert y.shape == (0, 4, 64)
    got = binding.block_norm_bwd(y, None, y, h, d["w1"], None, d["w2"])
    assert float(got[2].abs().max()) == 0.0 and got[3] is None and float(got[4].abs().max()) == 0.0
    g = heads(2, 5, 4, 32, "bf16", 3, True)
    assert binding.gated_norm_fwd(g["x"][:, :0], g["g"][:, :0], g["w"]).shape == (2, 0, 4, 32)
    assert float(binding.gated_norm_bwd(*(g[n][:, :0] for n in ("dy", "x", "g")), g["w"])[2].abs().max()) == 0.0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = binding.gated_norm_fwd(g["x"], g["g"], g["w"], stream=s)
    b = binding.block_norm_fwd(d["x"], d["res"], d["w1"], d["s"], d["w2"], stream=s)
    s.synchronize()
    assert torch.equal(a, binding.gated_norm_fwd(g["x"], g["g"], g["w"])) and torch.equal(b[0], want[0])


def test_refusals():
    g, d = heads(2, 5, 4, 32, "bf16", 3, True), rows(12, 64, "bf16", 1, 3)
    f, b = binding.gated_norm_fwd, binding.block_norm_fwd
    with pytest.raises(TypeError):
        f(g["x"].half(), g["g"])
    with pytest.raises(TypeError):
        f(g["x"], g["g"].float())
    with pytest.raises(TypeError):
        f(g["x"][0], g["g"][0])
    with pytest.raises(ValueError):
        f(g["x"], g["g"][:1])
    with pytest.raises(ValueError):
        f(g["x"], g["g"], g["w"][:8])
    with pytest.raises(TypeError):
        f(g["x"], g["g"], g["w"].bfloat16())
    with pytest.raises(ValueError):
        f(g["x"].transpose(2, 3), g["g"].transpose(2, 3))
    with pytest.raises(ValueError):
        f(g["x"], g["g"], y=g["x"])
    with pytest.raises(binding.GdnError):
        f(g["x"], g["g"], eps=-1.0)
    with pytest.raises(binding.GdnError):
        f(g["x"][..., :4].contiguous(), g["g"][..., :4].contiguous())
    with pytest.raises(binding.GdnError):
        binding.gated_norm_bwd(g["dy"], g["x"], g["g"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        b(d["x"], d["res"][:3])
    with pytest.raises(ValueError):
        b(d["x"], d["res"], scale=d["s"][:, :8])
    with pytest.raises(ValueError):
        b(d["x"][:11], d["res"][:11], scale=d["s"])
    with pytest.raises(TypeError):
        b(d["x"], d["res"].float())
    with pytest.raises(binding.GdnError):
        b(d["x"], d["res"], eps=float("nan"))
    with pytest.raises(binding.GdnError):
        b(d["x"][:, :4].contiguous(), d["res"][:, :4].contiguous())
    with pytest.raises(ValueError):
        binding.block_norm_bwd(d["dy"][:3], None, d["x"], d["x"])
