"""Linear attention with a decay for each head over prompts: the CUDA kernels
against the token recurrence in 64 bits.

Bounds, on max|x - ref| / max|ref|: the library's targets for outputs in the
tensors' type (1e-2 bf16, 1e-4 fp32).  The fp32 outputs of bf16 calls (states,
their gradients, dg) come from exact products of bf16 inputs with weights and
states kept to 16 bits of mantissa or more (relative 2^-16 = 1.5e-5 a term,
random over the terms) and fp32 sums: 1e-4 holds them with room."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, TOL_F32, ensure_lib, rel_err

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def inputs(B, H, Hk, T, Dk, Dv, dtype, seed, lens=None, per_head=False, g_scale=1 / 16, token_major=False):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    d = dict(q=unit(randn(B, Hk, T, Dk)), k=unit(randn(B, Hk, T, Dk)), v=randn(B, H, T, Dv), do=randn(B, H, T, Dv))
    d = {n: x.to(DT[dtype]) for n, x in d.items()}
    d["g"] = torch.nn.functional.logsigmoid(randn(H) if per_head else randn(B, H, T)) * g_scale
    n = B if lens is None else len(lens)
    d["s0"], d["dsf"] = 0.3 * randn(n, H, Dk, Dv), 0.3 * randn(n, H, Dk, Dv)
    d = {n: x.cuda() for n, x in d.items()}
    if token_major:
        for name in ("q", "k", "v", "do"):
            d[name] = d[name].transpose(1, 2).contiguous().transpose(1, 2)
    return d


def offsets(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


CASES = [  # B, H, Hk, T, Dk, Dv, lens, per head, token-major
    (1, 1, 1, 1, 128, 128, None, False, False),
    (2, 3, 3, 63, 128, 128, None, False, False),
    (1, 4, 2, 128, 128, 128, None, True, True),
    (2, 2, 1, 129, 128, 128, None, False, True),
    (1, 2, 2, 700, 128, 128, None, False, False),
    (1, 4, 2, 400, 128, 128, [1, 0, 127, 0, 129, 143, 0], False, True),
    (1, 2, 1, 300, 64, 64, [300], True, False),
    (1, 2, 2, 261, 64, 128, [64, 65, 132], False, True),
    (2, 2, 2, 190, 128, 64, None, False, False),
]


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("B,H,Hk,T,Dk,Dv,lens,per_head,token_major", CASES)
def test_forward(B, H, Hk, T, Dk, Dv, lens, per_head, token_major, states, dtype, simt):
    d = inputs(B, H, Hk, T, Dk, Dv, dtype, 11 + T, lens, per_head, token_major=token_major)
    s0 = d["s0"] if states else None
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=s0, output_final_state=states,
                                      cu_seqlens=None if lens is None else offsets(lens), scale=0.7, simt=simt)
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"], s0, lens, 0.7)
    assert o.stride() == d["v"].stride()
    assert rel_err(o, ro) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    if states:
        assert rel_err(sf, rs) <= 1e-5
    assert binding.device_error() == 0


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("B,H,Hk,T,Dk,Dv,lens,per_head,token_major", CASES)
def test_backward(B, H, Hk, T, Dk, Dv, lens, per_head, token_major, states, dtype, simt):
    d = inputs(B, H, Hk, T, Dk, Dv, dtype, 23 + T, lens, per_head, token_major=token_major)
    s0, dsf = (d["s0"], d["dsf"]) if states else (None, None)
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=s0, dfinal_state=dsf,
                                    cu_seqlens=None if lens is None else offsets(lens), scale=0.7, simt=simt)
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], s0, dsf, lens, 0.7)
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    for name, x, r in zip(("dq", "dk", "dv"), got, want):
        assert rel_err(x, r) <= tol, name
    assert rel_err(got[3], want[3]) <= 1e-4
    if states:
        assert rel_err(got[4], want[4]) <= 1e-5
    else:
        assert got[4] is None
    assert binding.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_against_differences(dtype):
    """Central differences of the 64-bit forward's loss along random directions."""
    d = inputs(1, 2, 1, 150, 128, 128, dtype, 5, [70, 80])
    lens, cu = [70, 80], offsets([70, 80])
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["s0"],
                                    dfinal_state=d["dsf"], cu_seqlens=cu)

    def loss(x):
        o, sf = ref.linattn(x["q"], x["k"], x["v"], x["g"], x["s0"], lens)
        return float((o * d["do"].double().cpu()).sum() + (sf * d["dsf"].double().cpu()).sum())

    base = {n: d[n].double().cpu() for n in ("q", "k", "v", "g", "s0")}
    gen = torch.Generator().manual_seed(1)
    for name, grad in zip(("q", "k", "v", "g", "s0"), got):
        u = torch.randn(base[name].shape, generator=gen, dtype=torch.float64)
        eps = 1e-6
        up, down = ({**base, name: base[name] + s * eps * u} for s in (1, -1))
        want, have = (loss(up) - loss(down)) / (2 * eps), float((grad.double().cpu() * u).sum())
        size = float((grad.double().cpu() * u).square().sum().sqrt())  # of a random sum like it
        # bf16 gradients carry 2^-9 of rounding a term, random over the terms; differences 1e-6 or less
        assert abs(have - want) <= (2e-2 if dtype == "bf16" else 1e-4) * max(size, 1e-12), name


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("f32", True)])
def test_tokens_of_no_sequence(dtype, simt):
    """Offsets that leave tokens out: zeros there, and what lies there (an
    infinity, a NaN) reaches nothing else."""
    lens, first, T = [100, 0, 37, 130], 21, 320
    d = inputs(1, 2, 1, T, 128, 128, dtype, 3, lens)
    end = first + sum(lens)
    for name in ("q", "k", "v", "do"):
        d[name][:, :, :first] = float("nan")
        d[name][:, :, end:] = float("inf")
    cu = offsets(lens, first)
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], output_final_state=True,
                                      cu_seqlens=cu, simt=simt)
    clean = {n: torch.nan_to_num(d[n].float(), 0.0, 0.0, 0.0) for n in ("q", "k", "v", "do")}
    ro, rs = ref.linattn(clean["q"], clean["k"], clean["v"], d["g"], d["s0"], lens, first=first)
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    assert float(o[:, :, :first].abs().max()) == 0.0 and float(o[:, :, end:].abs().max()) == 0.0
    assert rel_err(o, ro) <= tol and rel_err(sf, rs) <= 1e-5
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["s0"],
                                    dfinal_state=d["dsf"], cu_seqlens=cu, simt=simt)
    want = ref.linattn_bwd(clean["q"], clean["k"], clean["v"], d["g"], clean["do"], d["s0"], d["dsf"], lens, first=first)
    for x, r, t in zip(got, want, (tol, tol, tol, 1e-4, 1e-5)):
        assert rel_err(x, r) <= t
    for x in got[:3]:
        assert float(x[:, :, :first].abs().max()) == 0.0 and float(x[:, :, end:].abs().max()) == 0.0


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("bf16", True), ("f32", True)])
def test_one_sequence_does_not_reach_another(dtype, simt):
    """An infinity in one packed sequence leaves the others' outputs alone."""
    lens = [50, 90, 141]
    d = inputs(1, 2, 2, sum(lens), 128, 128, dtype, 9, lens)
    clean, _ = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=offsets(lens), simt=simt)
    for name in ("q", "k", "v"):
        d[name][:, :, 50:140] = float("inf")
    o, _ = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=offsets(lens), simt=simt)
    assert torch.equal(o[:, :, :50], clean[:, :, :50]) and torch.equal(o[:, :, 140:], clean[:, :, 140:])


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("bf16", True), ("f32", True)])
def test_decays_that_clear_the_state(dtype, simt):
    """g = -inf drops what came before it, as a new sequence does; strong
    decays over a whole chunk stay finite."""
    d = inputs(1, 2, 2, 300, 128, 128, dtype, 17)
    d["g"][:, :, 130] = float("-inf")
    d["g"][:, 1, 200:280] = -40.0
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], output_final_state=True, simt=simt)
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"])
    assert rel_err(o, ro) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    assert rel_err(sf, rs) <= 1e-5
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], simt=simt)
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"])
    for x, r in zip(got[:4], want):
        assert rel_err(x, r) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)


def test_split_and_resume():
    """A prompt in two calls, the first one's state going into the second."""
    d = inputs(1, 4, 2, 500, 128, 128, "bf16", 31)
    whole, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], output_final_state=True)
    cut = 213
    a, s1 = binding.linattn_chunk_fwd(*(d[n][:, :, :cut] for n in "qkvg"), output_final_state=True)
    b, s2 = binding.linattn_chunk_fwd(*(d[n][:, :, cut:] for n in "qkvg"), initial_state=s1, output_final_state=True)
    # the same exact products in another order and cut: bf16 outputs, fp32 states
    assert rel_err(torch.cat([a, b], 2), whole.double().cpu().numpy()) <= TOL_BF16
    assert rel_err(s2, sf.double().cpu().numpy()) <= 1e-5


def test_long_and_many_sequences():
    """A long row against the first and last sequences alone, and many short ones."""
    lens = [3000, 5] + [1] * 40 + [77, 2049]
    d = inputs(1, 2, 1, sum(lens), 128, 128, "bf16", 41, lens)
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], output_final_state=True,
                                      cu_seqlens=offsets(lens))
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"], d["s0"], lens)
    assert rel_err(o, ro) <= TOL_BF16 and rel_err(sf, rs) <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_calls_give_equal_bits(dtype):
    d = inputs(2, 4, 2, 333, 128, 128, dtype, 2)
    a = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"])
    b = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"])
    c = [binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"])[0] for _ in range(2)]
    assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4])) and torch.equal(*c)


def test_views_streams_and_expanded_inputs():
    """Slices of one projection, an expanded input, another stream."""
    B, H, T, D = 2, 4, 200, 128
    gen = torch.Generator().manual_seed(8)
    qkv = torch.randn(B, T, 3 * H, D, generator=gen).cuda().bfloat16()
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    g = -torch.rand(B, T, H, generator=gen).cuda().transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, _ = binding.linattn_chunk_fwd(q, k, v, g, scale=0.1, stream=s)
    s.synchronize()
    ro, _ = ref.linattn(q, k, v, g, scale=0.1)
    assert rel_err(o, ro) <= TOL_BF16
    one = k[:, :1].expand(B, H, T, D)
    o, _ = binding.linattn_chunk_fwd(q, one, v, g, scale=0.1)
    ro, _ = ref.linattn(q, one, v, g, scale=0.1)
    assert rel_err(o, ro) <= TOL_BF16
    got = binding.linattn_chunk_bwd(q, one, v, g, v, scale=0.1)
    want = ref.linattn_bwd(q, one, v, g, v, scale=0.1)
    for x, r in zip(got[:3], want):
        assert rel_err(x, r) <= TOL_BF16


def test_empty():
    d = inputs(2, 2, 2, 4, 64, 64, "bf16", 1)
    empty = [d[n][:, :, :0] for n in "qkvg"]
    o, sf = binding.linattn_chunk_fwd(*empty, initial_state=d["s0"], output_final_state=True)
    assert o.numel() == 0 and torch.equal(sf, d["s0"])
    got = binding.linattn_chunk_bwd(*empty, d["do"][:, :, :0], initial_state=d["s0"], dfinal_state=d["dsf"])
    assert torch.equal(got[4], d["dsf"])


def test_refusals():
    d = inputs(1, 2, 2, 16, 64, 64, "bf16", 1)
    f = binding.linattn_chunk_fwd
    with pytest.raises(TypeError):
        f(d["q"].cpu(), d["k"], d["v"], d["g"])
    with pytest.raises(TypeError):
        f(d["q"].half(), d["k"].half(), d["v"].half(), d["g"])
    with pytest.raises(TypeError):
        f(d["q"], d["k"].float(), d["v"], d["g"])
    with pytest.raises(TypeError):
        f(d["q"], d["k"], d["v"], d["g"].double())
    with pytest.raises(ValueError):
        f(d["q"], d["k"][:, :, :8], d["v"], d["g"])
    with pytest.raises(ValueError):
        f(d["q"], d["k"], d["v"], d["g"][:, :1])
    with pytest.raises(ValueError):
        f(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"][:, :1])
    with pytest.raises(ValueError):
        f(d["q"].transpose(2, 3), d["k"].transpose(2, 3), d["v"][:, :, :, :].transpose(2, 3), d["g"])
    with pytest.raises(ValueError):  # rows not 16-byte aligned
        wide = torch.zeros(1, 2, 16, 65, device="cuda", dtype=torch.bfloat16)
        f(wide[..., :64], d["k"], d["v"], d["g"])
    with pytest.raises(ValueError):  # Dk = 32
        f(d["q"][..., :32], d["k"][..., :32], d["v"], d["g"])
    with pytest.raises(ValueError):  # packed rows
        two = inputs(2, 2, 2, 16, 64, 64, "bf16", 1)
        f(two["q"], two["k"], two["v"], two["g"], cu_seqlens=offsets([16]))
    with pytest.raises(TypeError):
        f(d["q"], d["k"], d["v"], d["g"], cu_seqlens=offsets([16]).long())
    with pytest.raises(ValueError):  # three value heads, two key heads
        three = inputs(1, 3, 3, 16, 64, 64, "bf16", 1)
        f(d["q"], d["k"], three["v"], three["g"])
    with pytest.raises(binding.GdnError):
        f(d["q"], d["k"], d["v"], d["g"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), simt=True)
