"""The operators next to a mixer at the sizes where each launch takes the form of a full
machine: several rows a thread in the steps of a full decoding batch, several rows a CTA
in the norms, strips of many tokens with sequences' ends inside them in the
convolution.  Against 64 bits on the GPU; the bounds are those of the operators'
own tests, derived there."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_causal_conv import DT, close as conv_close
from tests.test_gpu_gated_norm import close as norm_close, heads, rows
from tests.test_gpu_ssm_scan import close as scan_close

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def generator(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, device="cuda")


def busy_slots(B, pages, seed):
    """A page for each row, some idle: -1, and numbers past the pool."""
    gen = torch.Generator().manual_seed(seed)
    slots = torch.randperm(pages, generator=gen)[:B].to(torch.int32)
    slots[3::11] = -1
    slots[5::17] = pages + 7
    return slots.cuda(), ((slots >= 0) & (slots < pages)).cuda()


def silu(x):
    return x / (1 + torch.exp(-x))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype,B,C,W", [("bf16", 157, 8192, 4), ("bf16", 311, 4096, 3), ("f32", 81, 8192, 4), ("f32", 158, 4096, 2),
                                         ("bf16", 999, 1288, 2)])
def test_convolution_steps_of_a_full_batch(dtype, B, C, W, in_place):
    """Rows that are no multiple of a thread's, idle ones among a thread's others."""
    randn = generator(B)
    x, w, bias = randn(B, C).to(DT[dtype]), randn(C, W), randn(C)
    pool = randn(B + 9, W - 1, C).to(DT[dtype])
    slots, on = busy_slots(B, B + 9, B)
    at = slots[on].long()
    seq = torch.cat([pool[at], x[on][:, None]], 1)
    want = torch.zeros(B, C, dtype=torch.float64, device="cuda")
    want[on] = silu((seq.double() * w.double().t()).sum(1) + bias.double())
    after = pool.clone()
    after[at] = seq[:, 1:]
    out = None if in_place else pool.clone()
    y = binding.causal_conv_step(x, w, pool, bias, slots=slots, window_out=out)
    conv_close(y, want.cpu(), dtype)
    assert torch.equal(pool if in_place else out, after)
    assert float(y[~on].float().abs().max()) == 0.0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype,B,Di,N", [("bf16", 157, 2048, 16), ("f32", 77, 2048, 16), ("bf16", 201, 1288, 32), ("f32", 310, 1024, 8),
                                          ("bf16", 65700, 8, 8), ("f32", 65537, 8, 32)])
def test_scan_steps_of_a_full_batch(dtype, B, Di, N, in_place):
    """As above, and more rows than one launch takes."""
    randn = generator(B)
    x, dt, z = (randn(B, Di).to(DT[dtype]) for _ in range(3))
    Bt, Ct = randn(B, N).to(DT[dtype]), randn(B, N).to(DT[dtype])
    A, D, bias = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * randn(Di, N)), randn(Di), randn(Di) - 2
    pool = randn(B + 9, Di, N)
    slots, on = busy_slots(B, B + 9, B)
    at = slots[on].long()
    wide = lambda t: t[on].double()  # noqa: E731
    step = torch.nn.functional.softplus(wide(dt) + bias.double(), threshold=1e9)
    h = torch.exp(step[..., None] * A.double()) * pool[at].double() + (step * wide(x))[..., None] * wide(Bt)[:, None]
    want = torch.zeros(B, Di, dtype=torch.float64, device="cuda")
    want[on] = ((h * wide(Ct)[:, None]).sum(-1) + D.double() * wide(x)) * silu(wide(z))
    before = pool.clone()
    out = None if in_place else pool.clone()
    y = binding.ssm_step(x, dt, A, Bt, Ct, pool, D=D, z=z, dt_bias=bias, slots=slots, state_out=out)
    got = pool if in_place else out
    scan_close(y, want.cpu(), dtype, 1e-5)
    scan_close(got[at], h.cpu(), "f32", 1e-5)
    free = torch.ones(B + 9, dtype=torch.bool, device="cuda")
    free[at] = False
    assert torch.equal(got[free], before[free]) and float(y[~on].float().abs().max()) == 0.0


def test_scan_steps_of_many_rows_without_slots():
    """Row b on page b, past what one launch takes."""
    randn, B = generator(1), 65600
    x, dt, Bt, Ct = (randn(B, 8).bfloat16() for _ in range(4))
    A, pool = -torch.rand(8, 8, device="cuda"), randn(B, 8, 8)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    out, other = torch.empty_like(pool), torch.empty_like(pool)
    a = binding.ssm_step(x, dt, A, Bt, Ct, pool, slots=slots, state_out=out)
    b = binding.ssm_step(x, dt, A, Bt, Ct, pool, state_out=other)
    assert torch.equal(a, b) and torch.equal(out, other)


def inverse_norm(u):
    return 1 / ((u * u).mean(-1, keepdim=True) + EPS).sqrt()


def norm_back(t, u):
    """The gradient of u where u inverse_norm(u) has the gradient t."""
    r = inverse_norm(u)
    return r * t - u * r ** 3 * (t * u).mean(-1, keepdim=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C,groups", [(5003, 2048, 1), (20001, 64, 0), (1505, 8192, 5), (1999, 4104, 1), (9000, 1000, 3),
                                        (12000, 256, 40)])
def test_many_rows_of_a_block(n, C, groups, dtype):
    """Several rows a CTA: the next row's loads while one is summed up, ends of a CTA's rows."""
    d = rows(n, C, dtype, n, groups)
    wide = {k: None if t is None else t.double() for k, t in d.items()}
    s = torch.ones(1, C, dtype=torch.float64, device="cuda") if groups == 0 else wide["s"].reshape(-1, C)
    by = lambda t: t.reshape(len(s), -1, C)  # noqa: E731
    y, h = binding.block_norm_fwd(d["x"], d["res"], d["w1"], d["s"], d["w2"], eps=EPS)
    n1 = wide["x"] * inverse_norm(wide["x"])
    wh = wide["res"] + (by(n1 * wide["w1"]) * s[:, None]).reshape(n, C)
    norm_close(h, wh.cpu(), dtype)
    norm_close(y, (wh * inverse_norm(wh) * wide["w2"]).cpu(), dtype)
    del wh
    dx, dres, dw1, ds, dw2 = binding.block_norm_bwd(d["dy"], d["dh"], d["x"], h, d["w1"], d["s"], d["w2"], eps=EPS)
    h64 = h.double()
    wres = wide["dh"] + norm_back(wide["dy"] * wide["w2"], h64)
    norm_close(dres, wres.cpu(), dtype)
    scaled = (by(wres) * s[:, None]).reshape(n, C)
    norm_close(dx, norm_back(scaled * wide["w1"], wide["x"]).cpu(), dtype)
    many = 1e-5 + n ** 0.5 * 2.0 ** -22
    norm_close(dw1, (scaled * n1).sum(0).cpu(), "f32", many)
    norm_close(dw2, (wide["dy"] * h64 * inverse_norm(h64)).sum(0).cpu(), "f32", many)
    if groups:
        norm_close(ds, by(wres * wide["w1"] * n1).sum(1).reshape(d["s"].shape).cpu(), "f32", many)
    else:
        assert ds is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shared,gate_first", [(True, False), (False, True)])
@pytest.mark.parametrize("B,T,H,D", [(2, 1001, 3, 512), (1, 1999, 2, 1024), (1, 1203, 3, 2048), (3, 333, 1, 4104), (1, 901, 2, 8192),
                                     (1, 5001, 5, 264)])
def test_many_tokens_of_wide_heads(B, T, H, D, shared, gate_first, dtype):
    """Heads whose threads span warps, several tokens a group of threads."""
    d = heads(B, T, H, D, dtype, D, shared, heads_first=True)
    x, g, dy, w = (d[n].double() for n in ("x", "g", "dy", "w"))
    s = 1 / (1 + torch.exp(-g))
    act, slope = g * s, s + g * s * (1 - s)
    u = x * act if gate_first else x
    n = u * inverse_norm(u)
    y = binding.gated_norm_fwd(d["x"], d["g"], d["w"], eps=EPS, gate_first=gate_first)
    norm_close(y, (n * w if gate_first else n * w * act).cpu(), dtype)
    dx, dg, dw = binding.gated_norm_bwd(d["dy"], d["x"], d["g"], d["w"], eps=EPS, gate_first=gate_first)
    t = dy if gate_first else dy * act
    du = norm_back(t * w, u)
    norm_close(dx, (du * act if gate_first else du).cpu(), dtype)
    norm_close(dg, (du * x * slope if gate_first else dy * n * w * slope).cpu(), dtype)
    norm_close(dw, (t * n).sum((0, 1, 2) if shared else (0, 1)).cpu(), "f32", 1e-5 + (B * T * H) ** 0.5 * 2.0 ** -22)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,cu", [(1024, [0, 71, 72, 73, 1000, 1007, 1008, 1024, 1031, 1031, 9001, 16384]),
                                  (2048, [5, 144, 145, 150, 288, 3000, 3002, 3003, 8191, 16000]),
                                  (1024, [0, 16384])])
def test_ends_inside_long_strips(C, cu, W, dtype):
    """Strips of 72 to 300 tokens: groups of tokens inside one sequence beside groups with ends, sequences that pass
    over a strip's end by less and more than the taps."""
    T, n_seq = 16384, len(cu) - 1
    randn = generator(C + W)
    x, dy = randn(1, T, C).to(DT[dtype]), randn(1, T, C).to(DT[dtype])
    win, dwin = randn(n_seq, W - 1, C).to(DT[dtype]), randn(n_seq, W - 1, C).to(DT[dtype])
    w, bias = randn(C, W), randn(C)
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = binding.causal_conv_fwd(x, w, bias, initial_window=win, output_final_window=True, cu_seqlens=offsets)
    got = binding.causal_conv_bwd(x, w, dy, bias, initial_window=win, dfinal_window=dwin, cu_seqlens=offsets)
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    wy, wx, ww, wb, wlast, wwin = zero(T, C), zero(T, C), zero(C, W), zero(C), zero(n_seq, W - 1, C), zero(n_seq, W - 1, C)
    w64 = w.double()
    for q, (a, b) in enumerate(zip(cu, cu[1:])):
        seq = torch.cat([win[q].double(), x[0, a:b].double()])
        back = zero(*seq.shape)
        back[b - a:] += dwin[q].double()
        if b > a:
            taps = [seq[j: j + b - a] for j in range(W)]
            z = sum(t * w64[:, j] for j, t in enumerate(taps)) + bias.double()
            s = 1 / (1 + torch.exp(-z))
            wy[a:b] = z * s
            dz = dy[0, a:b].double() * (s + z * s * (1 - s))
            wb += dz.sum(0)
            for j, t in enumerate(taps):
                ww[:, j] += (dz * t).sum(0)
                back[j: j + b - a] += dz * w64[:, j]
        wlast[q] = seq[b - a:]
        wx[a:b], wwin[q] = back[W - 1:], back[: W - 1]
    conv_close(y[0], wy.cpu(), dtype)
    assert torch.equal(last.double(), wlast)
    conv_close(got[0][0], wx.cpu(), dtype)
    conv_close(got[1], ww.cpu(), "f32", 8e-6 + T ** 0.5 * 2.0 ** -22)
    conv_close(got[2], wb.cpu(), "f32", 8e-6 + T ** 0.5 * 2.0 ** -22)
    conv_close(got[3], wwin.cpu(), dtype)
