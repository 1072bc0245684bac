"""The operators next to a mixer run together as a layer uses them: a state space
layer (norms around the block, short convolution, scan) and a linear-attention one
(convolution in front of q, k and v, gated norm behind the heads), served over
packed prompts and then token by token, and trained.  Every call is checked against
the 64-bit form of the values that it was given; what the calls carry from one to
the next (windows, states, pages) against the whole sequence's."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests import layer_reference, mixer_reference as ref
from tests.gpu_util import TOL_BF16, ensure_lib, rel_err
from tests.test_gpu_causal_conv import close

pytestmark = pytest.mark.gpu

C, N, W = 256, 16, 4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    proj = lambda a, b: (randn(a, b) / a ** 0.5).bfloat16()  # noqa: E731
    return dict(inp=proj(C, 2 * C), dbc=proj(C, C + 2 * N), out=proj(C, C), taps=randn(C, W) / 2, bias=0.1 * randn(C),
                A=-torch.arange(1, N + 1).cuda() * torch.exp(0.1 * randn(C, N)), D=randn(C), dt_bias=randn(C) - 3,
                pre=1 + 0.1 * randn(C), post=1 + 0.1 * randn(C), scale=0.5 + 0.1 * randn(C), nxt=1 + 0.1 * randn(C))


def block(w, x, res, conv, scan):
    """One state space block between two norms; `conv` and `scan` keep what they carry."""
    u, _, h = binding.rms_norm_fwd(x, w["pre"], residual=res)
    xz = u @ w["inp"]
    xs, z = xz[..., :C], xz[..., C:]
    xs = conv(xs)
    dbc = xs @ w["dbc"]
    y = scan(xs, dbc[..., :C], dbc[..., C:C + N], dbc[..., C + N:], z)
    o = y @ w["out"]
    return binding.block_norm_fwd(o, h, w["post"], w["scale"], w["nxt"])


def test_serving_a_state_space_layer():
    """Packed prompts, then tokens of each request: the tokens' outputs are those of one longer prompt."""
    w, lens, more = weights(1), [37, 5, 0, 130], 3
    gen = torch.Generator().manual_seed(2)
    rows = lambda n: torch.randn(n, C, generator=gen).bfloat16().cuda()  # noqa: E731
    xs, rs = [rows(n + more) for n in lens], [rows(n + more) for n in lens]

    def packed(take):
        offsets = torch.tensor([0] + torch.tensor([len(take(x)) for x in xs]).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        kept = {}

        def conv(x):
            y, kept["win"] = binding.causal_conv_fwd(x, w["taps"], w["bias"], output_final_window=True, cu_seqlens=offsets)
            return y

        def scan(x, dt, B, Cm, z):
            y, kept["state"] = binding.ssm_scan_fwd(x, dt, w["A"], B, Cm, D=w["D"], z=z, dt_bias=w["dt_bias"],
                                                    output_final_state=True, cu_seqlens=offsets)
            return y
        y, h = block(w, torch.cat([take(x) for x in xs])[None], torch.cat([take(r) for r in rs])[None], conv, scan)
        return y[0], h[0], kept, offsets

    _, _, kept, _ = packed(lambda x: x[:len(x) - more])
    full, full_h, ends, offsets = packed(lambda x: x)
    # the requests' pages: windows and states in pools, out of order, one page free
    slots = torch.tensor([4, 0, 3, 1], dtype=torch.int32, device="cuda")
    windows, states = torch.full((5, W - 1, C), 9.0, device="cuda").bfloat16(), torch.full((5, C, N), 9.0, device="cuda")
    windows[slots.long()], states[slots.long()] = kept["win"], kept["state"]
    for i in range(more):
        tok = torch.stack([x[len(x) - more + i] for x in xs])
        res = torch.stack([r[len(r) - more + i] for r in rs])
        y, h = block(w, tok, res, lambda x: binding.causal_conv_step(x, w["taps"], windows, w["bias"], slots=slots),
                     lambda x, dt, B, Cm, z: binding.ssm_step(x, dt, w["A"], B, Cm, states, D=w["D"], z=z, dt_bias=w["dt_bias"],
                                                              slots=slots))
        at = offsets[1:].long() - more + i
        # library products of other shapes may round their bf16 outputs otherwise
        assert rel_err(h, full_h[at].double().cpu().numpy()) <= TOL_BF16
        assert rel_err(y, full[at].double().cpu().numpy()) <= 2 * TOL_BF16
    assert rel_err(states[slots.long()], ends["state"].double().cpu().numpy()) <= 2 * TOL_BF16
    assert float(windows[2].float().min()) == 9.0 and float(states[2].min()) == 9.0


def test_training_a_state_space_layer():
    """A loss back through the block: each operator's gradient feeds the one before it."""
    w = weights(3)
    gen = torch.Generator().manual_seed(4)
    x, res, dy, dh = (torch.randn(2, 70, C, generator=gen).bfloat16().cuda() for _ in range(4))
    seen = {}

    def conv(x):
        seen["conv"] = x
        return binding.causal_conv_fwd(x, w["taps"], w["bias"])[0]

    def scan(x, dt, B, Cm, z):
        seen["scan"] = (x, dt, B, Cm, z)
        return binding.ssm_scan_fwd(x, dt, w["A"], B, Cm, D=w["D"], z=z, dt_bias=w["dt_bias"])[0]
    u, _, h0 = binding.rms_norm_fwd(x, w["pre"], residual=res)
    xz = u @ w["inp"]
    xs = conv(xz[..., :C])
    dbc = xs @ w["dbc"]
    y = scan(xs, dbc[..., :C], dbc[..., C:C + N], dbc[..., C + N:], xz[..., C:])
    o = y @ w["out"]
    _, h1 = binding.block_norm_fwd(o, h0, w["post"], w["scale"], w["nxt"])
    do, dres, dpost, dscale, dnxt = binding.block_norm_bwd(dy, dh, o, h1, w["post"], w["scale"], w["nxt"])
    xs, dt, B, Cm, z = seen["scan"]
    dyo = do @ w["out"].t()
    dxs, ddt, dA, dB, dC, dD, dz, dbias, _ = binding.ssm_scan_bwd(xs, dt, w["A"], B, Cm, dyo, D=w["D"], z=z, dt_bias=w["dt_bias"])
    dxs = dxs + torch.cat([ddt, dB, dC], -1) @ w["dbc"].t()
    dxc, dtaps, dcb, _ = binding.causal_conv_bwd(seen["conv"], w["taps"], dxs, w["bias"])
    du = torch.cat([dxc, dz], -1) @ w["inp"].t()
    dx, dpre = binding.rms_norm_bwd(du, h0, w["pre"], dresidual=dres)
    # against the same chain in 64 bits, each operator at the inputs that it was given
    leaf = ref.leaves(x=seen["conv"], w=w["taps"], b=w["bias"])
    got = ref.grads((ref.conv(leaf["x"], leaf["w"], leaf["b"])[0],), (ref.wide(dxs),), leaf)
    close(dxc, got["x"], "bf16")
    close(dtaps, got["w"], "f32", 1e-5)
    close(dcb, got["b"], "f32", 1e-5)
    leaf = ref.leaves(x=xs, dt=dt, A=w["A"], B=B, C=Cm, D=w["D"], z=z, bias=w["dt_bias"])
    got = ref.grads((ref.scan(*leaf.values())[0],), (ref.wide(dyo),), leaf)
    for t, n, dtype in ((dxs - torch.cat([ddt, dB, dC], -1) @ w["dbc"].t(), None, None), (ddt, "dt", "bf16"), (dA, "A", "f32"),
                        (dB, "B", "bf16"), (dC, "C", "bf16"), (dD, "D", "f32"), (dz, "z", "bf16"), (dbias, "bias", "f32")):
        if n:
            close(t, got[n], dtype, 1e-4)
    want = layer_reference.rms_norm_bwd(du, h0, w["pre"], dres)
    assert rel_err(dx, want[0].numpy()) <= TOL_BF16 and rel_err(dpre, want[1].numpy()) <= 1e-4
    assert all(bool(t.isfinite().all()) for t in (dpost, dscale, dnxt, dx))


def test_linear_attention_between_convolution_and_gated_norm():
    """q, k and v out of one convolution as views, the heads' output into the gated norm as it comes, and back."""
    H, D, T, lens = 4, 64, 90, [40, 1, 49]
    gen = torch.Generator().manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, gate = randn(1, T, 3 * H * D).bfloat16().cuda(), randn(1, T, H, D).bfloat16().cuda()
    taps, wn = (randn(3 * H * D, W) / 2).cuda(), (1 + 0.1 * randn(D)).cuda()
    g = torch.nn.functional.logsigmoid(randn(1, H, T) + 2).cuda()
    cu = torch.tensor([0, 40, 41, 90], dtype=torch.int32, device="cuda")
    mixed, _ = binding.causal_conv_fwd(x, taps, cu_seqlens=cu)
    close(mixed, ref.conv(ref.wide(x), ref.wide(taps), cu=cu.tolist())[0], "bf16")
    q, k, v = (t.unflatten(-1, (H, D)).transpose(1, 2) for t in mixed.split(H * D, -1))
    o, _ = binding.linattn_chunk_fwd(q, k, v, g, cu_seqlens=cu, scale=D ** -0.5)
    assert rel_err(o, layer_reference.linattn(q, k, v, g, None, lens, D ** -0.5)[0].numpy()) <= TOL_BF16
    heads = o.transpose(1, 2)
    y = binding.gated_norm_fwd(heads, gate, wn)
    close(y, ref.gated(ref.wide(heads), ref.wide(gate), ref.wide(wn)), "bf16", 1e-5)
    dy = randn(1, T, H, D).bfloat16().cuda()
    dheads, dgate, dwn = binding.gated_norm_bwd(dy, heads, gate, wn)
    dq, dk, dv, _, _ = binding.linattn_chunk_bwd(q, k, v, g, dheads.transpose(1, 2), cu_seqlens=cu, scale=D ** -0.5)
    dmixed = torch.cat([t.transpose(1, 2).flatten(2) for t in (dq, dk, dv)], -1)
    dx, dtaps, _, _ = binding.causal_conv_bwd(x, taps, dmixed, cu_seqlens=cu)
    leaf = ref.leaves(x=x, w=taps)
    got = ref.grads((ref.conv(leaf["x"], leaf["w"], cu=cu.tolist())[0],), (ref.wide(dmixed),), leaf)
    close(dx, got["x"], "bf16")
    close(dtaps, got["w"], "f32", 1e-5)
    assert dgate.shape == gate.shape and bool(dwn.isfinite().all())
