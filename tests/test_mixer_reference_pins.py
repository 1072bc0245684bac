"""The 64-bit forms that the mixer's kernels are tested against, pinned to something
else: torch's convolution, closed forms, and linear attention's recurrence."""
import torch

from tests import layer_reference, mixer_reference as ref

GEN = torch.Generator().manual_seed(7)


def randn(*s):
    return torch.randn(*s, generator=GEN, dtype=torch.float64)


def test_convolution_is_torchs():
    x, w, b = randn(2, 9, 5), randn(5, 4), randn(5)
    padded = torch.nn.functional.pad(x.transpose(1, 2), (3, 0))
    want = torch.nn.functional.conv1d(padded, w[:, None], b, groups=5).transpose(1, 2)
    y, win = ref.conv(x, w, b, act=False)
    assert torch.allclose(y, want, atol=1e-12) and torch.equal(win, x[:, -3:])
    assert torch.allclose(ref.conv(x, w, b)[0], torch.nn.functional.silu(want), atol=1e-12)


def test_windows_carry_a_sequence_on():
    x, w = randn(1, 11, 3), randn(3, 3)
    whole, last = ref.conv(x, w)
    a, win = ref.conv(x[:, :4], w)
    b, end = ref.conv(x[:, 4:], w, win=win)
    assert torch.allclose(torch.cat([a, b], 1), whole) and torch.equal(end, last)
    packed, wins = ref.conv(torch.cat([x, x], 1), w, cu=[0, 11, 11, 22], win=torch.zeros(3, 2, 3, dtype=torch.float64))
    assert torch.allclose(packed[:, 11:], whole) and torch.equal(wins[1], torch.zeros(2, 3, dtype=torch.float64))


def test_scan_of_one_state_is_linear_attention():
    """With one decay for all channels and states the state is k v^T, and the scan linear attention's recurrence."""
    T, Di, N = 12, 6, 8
    x, B, C = randn(1, T, Di), randn(1, T, N), randn(1, T, N)
    step = torch.rand(1, T, 1, generator=GEN, dtype=torch.float64).expand(1, T, Di)
    y, h = ref.scan(x, step, torch.full((Di, N), -0.7, dtype=torch.float64), B, C, soft=False)
    g = -0.7 * step[..., 0]
    o, S = layer_reference.linattn(C[:, None], B[:, None], (step * x)[:, None], g[:, None])
    assert torch.allclose(y, o[:, 0], atol=1e-12) and torch.allclose(h[0], S[0, 0].t(), atol=1e-12)


def test_scan_closed_forms():
    x, dt, B, C, A = randn(1, 1, 4), randn(1, 1, 4), randn(1, 1, 8), randn(1, 1, 8), -torch.rand(4, 8, generator=GEN, dtype=torch.float64)
    s0, D, z = randn(1, 4, 8), randn(4), randn(1, 1, 4)
    step = torch.nn.functional.softplus(dt[0, 0])
    h = torch.exp(step[:, None] * A) * s0[0] + (step * x[0, 0])[:, None] * B[0, 0]
    want = ((h @ C[0, 0]) + D * x[0, 0]) * torch.nn.functional.silu(z[0, 0])
    y, state = ref.scan(x, dt, A, B, C, D, z, s0=s0)
    assert torch.allclose(y[0, 0], want) and torch.allclose(state[0], h)
    zero = torch.zeros(1, 5, 4, dtype=torch.float64)
    y, state = ref.scan(zero, zero, A, B.expand(1, 5, 8), C.expand(1, 5, 8), s0=s0, soft=False)  # steps of 0 keep the state
    assert torch.allclose(state, s0) and torch.allclose(y[0, 4], s0[0] @ C[0, 0])


def test_norms():
    x, g, w = randn(1, 3, 2, 8), randn(1, 3, 2, 8), randn(8)
    n = torch.nn.functional.rms_norm(x, (8,), w, 1e-6)
    assert torch.allclose(ref.gated(x, g, w), n * torch.nn.functional.silu(g))
    assert torch.allclose(ref.gated(x, g, w, sigmoid=True), n * torch.sigmoid(g))
    u = x * torch.nn.functional.silu(g)
    assert torch.allclose(ref.gated(x, g, w, first=True), torch.nn.functional.rms_norm(u, (8,), w, 1e-6))
    a, r, s = randn(6, 8), randn(6, 8), randn(2, 8)
    y, h = ref.block(a, r, w, s, w)
    want = r + s.repeat_interleave(3, 0) * torch.nn.functional.rms_norm(a, (8,), w, 1e-6)
    assert torch.allclose(h, want) and torch.allclose(y, torch.nn.functional.rms_norm(want, (8,), w, 1e-6))
