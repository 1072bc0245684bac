"""The short convolution against 64 bits.  A value is rounded once, from fp32:
half a step of its type (bf16 2^-8, fp32 2^-24) and the fp32 arithmetic before,
at most 8 roundings of terms that add up to S (W products, bias, SiLU or its
slope): 8 * 2^-24 S, and S <= 16 times the largest output here: 8e-6 of it.
Sums over n tokens add n 2^-24 of their terms' sum."""
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


def close(got, want, dtype, slack=8e-6):
    got = got.double().cpu()
    assert got.shape == want.shape and bool(got.isfinite().all())
    err = (got - want).abs() - HALF[dtype] * want.abs()
    assert float(err.max() if err.numel() else 0) <= slack * max(float(want.abs().max() if want.numel() else 0), 1e-30)


def inputs(B, T, C, W, dtype, seed, n_seq=None, bias=True, states=True):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if n_seq is None else n_seq
    d = dict(x=randn(B, T, C), dy=randn(B, T, C), win=randn(n, W - 1, C), dwin=randn(n, W - 1, C))
    d = {k: t.to(DT[dtype]).cuda() for k, t in d.items()}
    d["w"], d["b"] = randn(C, W).cuda(), randn(C).cuda() if bias else None
    if not states:
        d["win"] = d["dwin"] = None
    return d


def check(d, dtype, cu=None, act=True):
    offsets = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, win = binding.causal_conv_fwd(d["x"], d["w"], d["b"], initial_window=d["win"], output_final_window=True,
                                     cu_seqlens=offsets, silu=act)
    leaf = ref.leaves(x=d["x"], w=d["w"], b=d["b"], win=d["win"])
    wy, wwin = ref.conv(leaf["x"], leaf["w"], leaf["b"], leaf["win"], cu, act)
    close(y, wy.detach(), dtype)
    assert torch.equal(win.double().cpu(), wwin.detach())  # windows are moved, not computed
    got = binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"],
                                  cu_seqlens=offsets, silu=act)
    want = ref.grads((wy, wwin), (ref.wide(d["dy"]), ref.wide(d["dwin"])), leaf)
    n = d["x"].shape[0] * d["x"].shape[1]
    close(got[0], want["x"], dtype)
    close(got[1], want["w"], "f32", 8e-6 + n ** 0.5 * 2.0 ** -22)
    if d["b"] is not None:
        close(got[2], want["b"], "f32", 8e-6 + n ** 0.5 * 2.0 ** -22)
    else:
        assert got[2] is None
    if d["win"] is not None:
        close(got[3], want["win"], dtype)
    else:
        assert got[3] is None
    again = binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"],
                                    cu_seqlens=offsets, silu=act)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (2, 2, 24), (1, 3, 8), (3, 5, 40), (1, 9, 1000), (2, 33, 256), (1, 130, 72)])
def test_rows(B, T, C, W, dtype):
    check(inputs(B, T, C, W, dtype, T + C), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bias,states,act", [(False, True, True), (True, False, True), (False, False, False)])
def test_options(bias, states, act, dtype):
    check(inputs(2, 21, 64, 4, dtype, 3, bias=bias, states=states), dtype, act=act)


PACKS = [[0, 1, 1, 3, 6, 30], [0, 0, 30], [0, 30, 30], [5, 7, 20], [0, 8, 16, 24, 30], [0, 7, 9, 10, 11, 30], [30, 30], [0, 0],
         [-4, 3, 40], [2, 2, 2, 5]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("cu", PACKS)
def test_packs(cu, states, W, dtype):
    """Lengths of none to a few, tokens before and behind them all, offsets outside the row."""
    check(inputs(1, 30, 40, W, dtype, len(cu), n_seq=len(cu) - 1, states=states), dtype, cu)


def test_offsets_out_of_order_stay_in_bounds():
    d = inputs(1, 30, 40, 4, "bf16", 1, n_seq=4)
    for cu in ([9, 3, 25, 1, 30], [30, 20, 10, 5, 0], [-7, 99, 4, -1, 2]):
        offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        y, win = binding.causal_conv_fwd(d["x"], d["w"], d["b"], initial_window=d["win"], output_final_window=True,
                                         cu_seqlens=offsets)
        binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"],
                                cu_seqlens=offsets)
        torch.cuda.synchronize()
        assert y.shape == d["x"].shape and win.shape == d["win"].shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_projection(dtype):
    d = inputs(2, 37, 48, 4, dtype, 5)
    both = torch.randn(2, 40, 128, device="cuda").to(DT[dtype])
    both[:, :37, 64:112] = d["x"]
    x = both[:, :37, 64:112]
    dys = torch.zeros(2, 37, 64, device="cuda", dtype=DT[dtype])
    dys[..., 16:64] = d["dy"]
    y, _ = binding.causal_conv_fwd(x, d["w"], d["b"])
    assert torch.equal(y, binding.causal_conv_fwd(d["x"], d["w"], d["b"])[0])
    got = binding.causal_conv_bwd(x, d["w"], dys[..., 16:64], d["b"])
    want = binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"])
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    room = torch.full((2, 37, 96), 7.0, device="cuda", dtype=DT[dtype])
    binding.causal_conv_fwd(x, d["w"], d["b"], y=room[..., 32:80])
    assert torch.equal(room[..., 32:80], y) and float(room[..., :32].min()) == 7.0 and float(room[..., 80:].max()) == 7.0


def test_long_rows_cut_into_strips():
    """Strips meet: a long row against the same row in parts."""
    d = inputs(1, 40000, 16, 4, "bf16", 2)
    y, win = binding.causal_conv_fwd(d["x"], d["w"], d["b"], initial_window=d["win"], output_final_window=True)
    parts, w = [], d["win"]
    for t in range(0, 40000, 9999):
        o, w = binding.causal_conv_fwd(d["x"][:, t: t + 9999], d["w"], d["b"], initial_window=w, output_final_window=True)
        parts.append(o)
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(w, win)
    dx, dw, db, dwin = binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"])
    x, dy = d["x"].double(), d["dy"].double()
    rows = torch.cat([d["win"].double(), x], 1)[0]
    taps = rows.unfold(0, 4, 1)
    z = (taps * d["w"].double()).sum(-1) + d["b"].double()
    s = torch.sigmoid(z)
    dz = dy[0] * s * (1 + z * (1 - s))
    close(dw, (dz[..., None] * taps).sum(0).cpu(), "f32", 40000 ** 0.5 * 2.0 ** -22)
    close(db, dz.sum(0).cpu(), "f32", 40000 ** 0.5 * 2.0 ** -22)
    back = torch.zeros_like(rows)
    back[-3:] += d["dwin"][0].double()
    for j in range(4):
        back[j: j + 40000] += dz * d["w"][:, j].double()
    close(dx[0], back[3:].cpu(), "bf16")
    close(dwin[0], back[:3].cpu(), "bf16")


def test_differences():
    d = inputs(1, 12, 8, 4, "f32", 8)
    got = binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"])
    base = {n: ref.wide(d[n]) for n in ("x", "w", "b", "win")}

    def loss(**kw):
        a = {**base, **kw}
        y, win = ref.conv(a["x"], a["w"], a["b"], a["win"])
        return float((y * ref.wide(d["dy"])).sum() + (win * ref.wide(d["dwin"])).sum())
    gen = torch.Generator().manual_seed(1)
    for n, g in zip(("x", "w", "b", "win"), got):
        u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        want = (loss(**{n: base[n] + 1e-6 * u}) - loss(**{n: base[n] - 1e-6 * u})) / 2e-6
        assert abs(float((g.double().cpu() * u).sum()) - want) <= 1e-4 * float((g.double().cpu() * u).square().sum().sqrt())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 8), (5, 40), (33, 1000)])
def test_steps(B, C, W, dtype):
    """Steps follow the prompt: T tokens one at a time, in place and into another pool; idle rows and pages stay."""
    T = 5
    d = inputs(B, T, C, W, dtype, B + C)
    want, last = ref.conv(ref.wide(d["x"]), ref.wide(d["w"]), ref.wide(d["b"]), ref.wide(d["win"]))
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).cuda()
    pool = torch.randn(B + 3, W - 1, C, device="cuda").to(DT[dtype])
    pool[slots.long()] = d["win"]
    idle = pool.clone()
    for t in range(T):
        if t % 2:
            other = pool.clone()
            y = binding.causal_conv_step(d["x"][:, t], d["w"], pool, d["b"], slots=slots, window_out=other)
            pool = other
        else:
            y = binding.causal_conv_step(d["x"][:, t], d["w"], pool, d["b"], slots=slots)
        close(y, want[:, t], dtype)
    assert torch.equal(pool[slots.long()].double().cpu(), last)
    free = [s for s in range(B + 3) if s not in slots.tolist()]
    assert torch.equal(pool[free], idle[free])
    gone = torch.full_like(slots, -1)
    gone[0] = 99999
    before = pool.clone()
    y = binding.causal_conv_step(d["x"][:, 0], d["w"], pool, d["b"], slots=gone)
    assert float(y.float().abs().max()) == 0.0 and torch.equal(pool, before)


def test_bad_values_stay_in_their_channel_and_sequence():
    d = inputs(1, 40, 16, 4, "bf16", 4, n_seq=2, states=False)
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    clean, _ = binding.causal_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=cu)
    d["x"][0, 18, 3] = float("nan")
    d["x"][0, 30, 5] = float("-inf")
    y, win = binding.causal_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=cu, output_final_window=True)
    touched = torch.zeros(40, 16, dtype=torch.bool)
    touched[18:20, 3] = True
    touched[30:34, 5] = True
    assert torch.equal(y[0].cpu()[~touched], clean[0].cpu()[~touched])
    assert bool(y[0, 18:20, 3].isnan().all()) and bool(win[0, 1, 3].isnan())


def test_empty_stream_and_refusals():
    d = inputs(2, 10, 16, 4, "bf16", 1)
    f, g = binding.causal_conv_fwd, binding.causal_conv_bwd
    y, win = f(d["x"][:, :0], d["w"], d["b"], initial_window=d["win"], output_final_window=True)
    assert y.shape == (2, 0, 16) and torch.equal(win, d["win"])
    got = g(d["x"][:, :0], d["w"], d["dy"][:, :0], d["b"], initial_window=d["win"], dfinal_window=d["dwin"])
    assert float(got[1].abs().max()) == 0.0 and float(got[2].abs().max()) == 0.0 and torch.equal(got[3], d["dwin"])
    assert binding.causal_conv_step(d["x"][:0, 0], d["w"], d["win"], d["b"]).shape == (0, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = f(d["x"], d["w"], d["b"])[0]
    got = f(d["x"], d["w"], d["b"], stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(TypeError):
        f(d["x"].half(), d["w"])
    with pytest.raises(TypeError):
        f(d["x"], d["w"].bfloat16())
    with pytest.raises(TypeError):
        f(d["x"][0], d["w"])
    with pytest.raises(ValueError):
        f(d["x"], d["w"][:8])
    with pytest.raises(ValueError):
        f(d["x"], d["w"], initial_window=d["win"][:1])
    with pytest.raises(TypeError):
        f(d["x"], d["w"], initial_window=d["win"].float())
    with pytest.raises(ValueError):
        f(d["x"].transpose(1, 2), d["w"][:10])
    with pytest.raises(ValueError):
        f(d["x"], d["w"], cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        f(d["x"], d["w"], y=d["x"])
    with pytest.raises(ValueError):
        f(d["x"], d["w"], y=torch.empty(1, 10, 16, device="cuda", dtype=torch.bfloat16).expand(2, 10, 16))
    with pytest.raises(binding.GdnError):
        f(d["x"], torch.zeros(16, 5, device="cuda"))
    with pytest.raises(binding.GdnError):
        f(d["x"][..., :4].contiguous(), d["w"][:4])
    with pytest.raises(ValueError):
        g(d["x"], d["w"], d["dy"][:, :5])
    with pytest.raises(binding.GdnError):
        g(d["x"], d["w"], d["dy"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        binding.causal_conv_step(d["x"][:, 0], d["w"], d["win"][:1])
    with pytest.raises(ValueError):
        binding.causal_conv_step(d["x"][:, 0], d["w"], d["win"], slots=torch.zeros(3, dtype=torch.int32, device="cuda"))
