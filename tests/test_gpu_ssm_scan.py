"""The selective state space scan against 64 bits.  A decay is off by 2^-22 at
most (an exponential of two units, its argument), a state over T tokens by T 2^-22
of its largest: with T up to 400, 1e-4 of the largest value holds fp32 values and
sums; bf16 values add half a step, 2^-8 of themselves."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import mixer_reference as ref
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "bias", "s0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def close(got, want, dtype, slack=1e-4):
    got = got.double().cpu()
    assert got.shape == want.shape and bool(got.isfinite().all())
    err = (got - want).abs() - HALF[dtype] * want.abs()
    assert float(err.max() if err.numel() else 0) <= slack * max(float(want.abs().max() if want.numel() else 0), 1e-30)


def inputs(B, T, Di, N, dtype, seed, n_seq=None, gate=True, skip=True, bias=True, states=True, soft=True):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if n_seq is None else n_seq
    d = dict(x=randn(B, T, Di), dt=randn(B, T, Di) - 2 if soft else torch.rand(B, T, Di, generator=gen) / 4, B=randn(B, T, N),
             C=randn(B, T, N), z=randn(B, T, Di) if gate else None, dy=randn(B, T, Di))
    d = {k: None if t is None else t.to(DT[dtype]).cuda() for k, t in d.items()}
    d["A"] = -(torch.arange(1, N + 1) * torch.exp(0.2 * randn(Di, N))).cuda()
    d["D"] = randn(Di).cuda() if skip else None
    # without softplus the bias is a step's part: a negative one of a half grows a state by e^8 a token, past fp32 after 12
    d["bias"] = (0.5 * (randn(Di) if soft else randn(Di).abs())).cuda() if bias else None
    d["s0"], d["dsf"] = (randn(n, Di, N).cuda(), randn(n, Di, N).cuda()) if states else (None, None)
    return d


def forward(d, cu=None, soft=True, **kw):
    return binding.ssm_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], dt_bias=d["bias"],
                                initial_state=d["s0"], output_final_state=True, cu_seqlens=cu, softplus=soft, **kw)


def backward(d, cu=None, soft=True, **kw):
    got = binding.ssm_scan_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], D=d["D"], z=d["z"], dt_bias=d["bias"],
                               initial_state=d["s0"], dfinal_state=d["dsf"], cu_seqlens=cu, softplus=soft, **kw)
    return dict(zip(NAMES, got))


def check(d, dtype, cu=None, soft=True):
    offsets = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    leaf = ref.leaves(**{n: d[n] for n in NAMES})
    wy, ws = ref.scan(*leaf.values(), cu=cu, soft=soft)
    y, state = forward(d, offsets, soft)
    close(y, wy.detach(), dtype)
    close(state, ws.detach(), "f32")
    want = ref.grads((wy, ws), (ref.wide(d["dy"]), ref.wide(d["dsf"])), leaf)
    got = backward(d, offsets, soft)
    order = dict(zip(("x", "dt", "A", "B", "C", "D", "z", "bias", "s0"), NAMES))
    for n in order:
        if want[n] is None:
            assert got[n] is None, n
        else:
            close(got[n], want[n], dtype if n in ("x", "dt", "B", "C", "z") else "f32")
    again = backward(d, offsets, soft)
    assert all(got[n] is again[n] or torch.equal(got[n], again[n]) for n in NAMES)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,T,Di", [(1, 1, 8), (2, 2, 24), (1, 7, 8), (1, 8, 136), (2, 9, 40), (1, 33, 264), (1, 130, 72),
                                    (3, 66, 16)])
def test_rows(B, T, Di, N, dtype):
    check(inputs(B, T, Di, N, dtype, T + Di), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", ["gate", "skip", "bias", "states", "soft", "all"])
def test_options(off, dtype):
    soft = off not in ("soft", "all")
    kw = {n: False for n in ("gate", "skip", "bias", "states") if off in (n, "all")}
    check(inputs(2, 21, 64, 16, dtype, 3, soft=soft, **kw), dtype, soft=soft)


PACKS = [[0, 1, 1, 3, 6, 90], [0, 0, 90], [0, 90, 90], [5, 7, 80], [0, 8, 16, 64, 90], [0, 63, 64, 65, 66, 90], [90, 90], [0, 0],
         [-4, 3, 140], [2, 2, 2, 5], [0, 70, 71, 90]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("cu", PACKS)
def test_packs(cu, states, dtype):
    """Lengths of none to a few, tokens before and behind them all, starts inside and at the ends of tiles and chunks."""
    check(inputs(1, 90, 40, 16, dtype, len(cu), n_seq=len(cu) - 1, states=states), dtype, cu)


@pytest.mark.parametrize("N", [8, 32])
def test_packs_of_other_states(N):
    check(inputs(1, 90, 72, N, "f32", N, n_seq=4), "f32", [0, 13, 40, 41, 90])


def test_tokens_of_no_sequence_may_be_anything():
    """NaN in tokens before and behind the sequences reaches nothing."""
    d = inputs(1, 90, 40, 16, "f32", 1, n_seq=2)
    cu = torch.tensor([6, 40, 75], dtype=torch.int32, device="cuda")
    clean = (*forward(d, cu), *backward(d, cu).values())
    for n in ("x", "dt", "B", "C", "z", "dy"):
        d[n][0, :6] = float("nan")
        d[n][0, 75:] = float("inf")
    dirty = (*forward(d, cu), *backward(d, cu).values())
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert float(dirty[0][0, :6].abs().max()) == 0.0 and float(dirty[0][0, 75:].abs().max()) == 0.0


def test_offsets_out_of_order_stay_in_bounds():
    d = inputs(1, 200, 40, 16, "bf16", 1, n_seq=4)
    for cu in ([9, 3, 125, 1, 200], [200, 120, 60, 5, 0], [-7, 299, 4, -1, 2]):
        offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        forward(d, offsets)
        backward(d, offsets)
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_projections(dtype):
    d = inputs(2, 37, 48, 16, dtype, 5)
    xz = torch.cat([d["x"], d["z"]], -1)
    proj = torch.cat([torch.zeros_like(d["B"])[..., :8], d["B"], d["C"]], -1)
    wide = torch.zeros(2, 37, 64, device="cuda", dtype=DT[dtype])
    wide[..., 8:56] = d["dy"]
    s = dict(d, x=xz[..., :48], z=xz[..., 48:], B=proj[..., 8:24], C=proj[..., 24:], dy=wide[..., 8:56])
    assert all(torch.equal(a, b) for a, b in zip(forward(s), forward(d)))
    a, b = backward(s), backward(d)
    assert all(torch.equal(a[n], b[n]) for n in NAMES)
    room = torch.full((2, 37, 96), 7.0, device="cuda", dtype=DT[dtype])
    y, _ = forward(s, y=room[..., 32:80])
    assert torch.equal(y, forward(d)[0]) and float(room[..., :32].min()) == 7.0 and float(room[..., 80:].max()) == 7.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Di,N", [(64, 16, 2048, 16), (28, 64, 2040, 16), (3, 608, 2048, 16), (56, 40, 2040, 8), (30, 17, 1000, 32)])
def test_full_machine(B, T, Di, N, dtype):
    """Rows and channels that fill the SMs: whole rows, rows of two chunks, of more chunks than are joined in place."""
    d = inputs(B, T, Di, N, dtype, T)
    wide = {n: ref.wide(d[n]) for n in NAMES}
    want, last = ref.scan(*wide.values())
    y, state = forward(d)
    close(y, want, dtype, max(1e-4, T * 2.0 ** -22))
    close(state, last, "f32", max(1e-4, T * 2.0 ** -22))


@pytest.mark.parametrize("B,T,Di", [(1, 5000, 64), (2, 1500, 256), (20, 300, 2048)])
def test_long_rows(B, T, Di):
    """Cut rows against the same rows in parts: states carry on, and so do their gradients."""
    d = inputs(B, T, Di, 16, "f32", 2)
    y, state = forward(d)
    got = backward(d)
    cuts = [0, T // 3 + 1, T // 2, T]
    states, outs = [d["s0"]], []
    part = lambda i: {n: t[:, cuts[i]: cuts[i + 1]] if n in ("x", "dt", "B", "C", "z", "dy") else t for n, t in d.items()}  # noqa: E731
    for i in range(3):
        o, s = forward(dict(part(i), s0=states[-1]))
        outs.append(o)
        states.append(s)
    close(y, torch.cat(outs, 1).double().cpu(), "f32", T * 2.0 ** -22)
    close(state, states[-1].double().cpu(), "f32", T * 2.0 ** -22)
    dsf, tokens, sums = d["dsf"], {n: [] for n in ("x", "dt", "B", "C", "z")}, {n: 0 for n in ("A", "D", "bias")}
    for i in (2, 1, 0):
        g = backward(dict(part(i), s0=states[i], dsf=dsf))
        dsf = g["s0"]
        for n in tokens:
            tokens[n].insert(0, g[n])
        for n in sums:
            sums[n] = sums[n] + g[n].double().cpu()
    for n in tokens:
        close(got[n], torch.cat(tokens[n], 1).double().cpu(), "f32", T * 2.0 ** -22)
    for n in sums:
        close(got[n], sums[n], "f32", T * 2.0 ** -22)
    close(got["s0"], dsf.double().cpu(), "f32", T * 2.0 ** -22)


def test_differences():
    d = inputs(1, 12, 8, 8, "f32", 8)
    got = backward(d)
    base = {n: ref.wide(d[n]) for n in NAMES}

    def loss(**kw):
        y, s = ref.scan(*{**base, **kw}.values())
        return float((y * ref.wide(d["dy"])).sum() + (s * ref.wide(d["dsf"])).sum())
    gen = torch.Generator().manual_seed(1)
    for n in NAMES:
        u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss(**{n: base[n] + 1e-6 * u}) - loss(**{n: base[n] - 1e-6 * u})) / 2e-6
        assert abs(float((got[n].double().cpu() * u).sum()) - want) <= 1e-4 * float((got[n].double().cpu() * u).square().sum().sqrt()), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("B,Di", [(1, 8), (5, 40), (33, 1000)])
def test_steps(B, Di, N, dtype):
    """Steps follow the prompt; idle rows give 0 and their pages stay."""
    T = 4
    d = inputs(B, T, Di, N, dtype, B + Di)
    want, last = ref.scan(*(ref.wide(d[n]) for n in NAMES))
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).cuda()
    pool = torch.randn(B + 3, Di, N, device="cuda")
    pool[slots.long()] = d["s0"]
    start = pool.clone()
    for t in range(T):
        out = pool.clone() if t % 2 else None
        y = binding.ssm_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], pool, D=d["D"], z=d["z"][:, t],
                             dt_bias=d["bias"], slots=slots, state_out=out)
        pool = pool if out is None else out
        close(y, want[:, t], dtype, 1e-5)
    close(pool[slots.long()], last, "f32", 1e-5)
    free = [s for s in range(B + 3) if s not in slots.tolist()]
    assert torch.equal(pool[free], start[free])
    gone = torch.full_like(slots, -1)
    gone[0] = 1 << 30
    before = pool.clone()
    y = binding.ssm_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], pool, slots=gone)
    assert float(y.float().abs().max()) == 0.0 and torch.equal(pool, before)


def test_extreme_steps():
    """Steps of 0 keep the state, huge ones clear it, and neither gives NaN."""
    d = inputs(1, 20, 16, 8, "f32", 4)
    d["dt"][0, 5] = -1e30   # softplus 0
    d["dt"][0, 11] = 1e4    # every decay 0
    d["x"][0, 11] = 0.0
    check(d, "f32")
    d["dt"][0, 5] = float("-inf")
    y, s = forward(d)
    assert bool(y.isfinite().all()) and bool(s.isfinite().all())


def test_bad_values_stay_in_their_channel_and_sequence():
    d = inputs(1, 80, 16, 8, "f32", 4, n_seq=2)
    cu = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    clean, cs = forward(d, cu)
    d["x"][0, 30, 3] = float("nan")
    d["dt"][0, 50, 5] = float("inf")
    y, s = forward(d, cu)
    touched = torch.zeros(80, 16, dtype=torch.bool)
    touched[30:40, 3] = True
    touched[50:, 5] = True
    assert torch.equal(y[0].cpu()[~touched], clean[0].cpu()[~touched]) and bool(y[0, 30:40, 3].isnan().all())
    d["x"][0, 30, 3] = 0.0
    d["B"][0, 60, 2] = float("nan")
    y, _ = forward(d, cu)
    assert bool(y[0, :40].isfinite().all()) and bool(y[0, 60:].isnan().all())


def test_empty_stream_and_refusals():
    d = inputs(2, 10, 16, 8, "bf16", 1)
    cut = lambda t: None if t is None else t[:, :0]  # noqa: E731
    e = {n: cut(t) if n in ("x", "dt", "B", "C", "z", "dy") else t for n, t in d.items()}
    y, s = forward(e)
    assert y.shape == (2, 0, 16) and torch.equal(s, d["s0"])
    g = backward(e)
    assert torch.equal(g["s0"], d["dsf"]) and float(g["A"].abs().max()) == 0.0 and float(g["D"].abs().max()) == 0.0
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = (*forward(d), *backward(d).values())
    got = (*forward(d, stream=st), *backward(d, stream=st).values())
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a = [d[n] for n in ("x", "dt", "A", "B", "C")]
    f = binding.ssm_scan_fwd

    def swapped(i, t):
        return [t if j == i else x for j, x in enumerate(a)]
    for i in (0, 1, 3, 4):
        with pytest.raises(TypeError):
            f(*swapped(i, a[i].half()))
        with pytest.raises((TypeError, ValueError)):
            f(*swapped(i, a[i][:, :5]))
    with pytest.raises(TypeError):
        f(*swapped(2, a[2].bfloat16()))
    with pytest.raises(ValueError):
        f(*swapped(2, a[2][:8]))
    with pytest.raises(ValueError, match="sizes rejected"):
        f(a[0], a[1], torch.zeros(16, 4, device="cuda"), a[3][..., :4].contiguous(), a[4][..., :4].contiguous())
    with pytest.raises(ValueError):
        f(*a, initial_state=d["s0"][:1])
    with pytest.raises(ValueError):
        f(*a, y=d["x"])
    with pytest.raises(ValueError):
        f(*a, z=d["z"][..., :8])
    with pytest.raises(ValueError):
        f(*a, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, device="cuda"))
    with pytest.raises(binding.GdnError):
        binding.ssm_scan_bwd(*a, d["dy"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        binding.ssm_scan_bwd(*a, d["dy"][:, :3])
    row = [d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0]]
    with pytest.raises(ValueError):
        binding.ssm_step(*row, d["s0"][:1])
    with pytest.raises(TypeError):
        binding.ssm_step(*row, d["s0"].bfloat16())
