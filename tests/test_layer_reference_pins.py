"""The 64-bit forms that the layer operators are tested against, pinned: their
backward passes against automatic differentiation of their forward ones, the
prompt against single steps, and worked values."""
import math

import torch

from tests import layer_reference as ref

CLOSE = dict(rtol=1e-12, atol=1e-12)  # 64-bit sums of a few hundred terms


def draw(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


def attention(q, k, v, g, s0, lens, scale):
    """ref.linattn as differentiable matrices: every pair's decay from the gates between."""
    B, H, T, _ = v.shape
    rep = H // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    outs, ends = [], []
    for s, (row, t0, n) in enumerate(ref.sequences(B, T, lens)):
        cum = torch.cat([torch.zeros(H, 1, dtype=torch.float64), g[row, :, t0:t0 + n].cumsum(-1)], 1)
        w = (cum[:, 1:, None] - cum[:, None, 1:]).tril().exp().tril()
        a = q[row, :, t0:t0 + n] @ k[row, :, t0:t0 + n].transpose(1, 2) * w
        o = a @ v[row, :, t0:t0 + n] + cum[:, 1:, None].exp() * (q[row, :, t0:t0 + n] @ s0[s])
        last = (cum[:, -1:] - cum[:, 1:]).exp()
        ends.append(cum[:, -1, None, None].exp() * s0[s] + (last[..., None] * k[row, :, t0:t0 + n]).transpose(1, 2) @ v[row, :, t0:t0 + n])
        outs.append(scale * o)
    return torch.cat(outs, 1)[None] if lens is not None else torch.stack(outs), torch.stack(ends)


def test_prompt_and_its_gradients():
    for B, lens in ((2, None), (1, [5, 0, 7, 1])):
        T, H, Hk, Dk, Dv = 13 if lens else 6, 4, 2, 3, 5
        q, k, v, g = draw(B, Hk, T, Dk, seed=1), draw(B, Hk, T, Dk, seed=2), draw(B, H, T, Dv, seed=3), -draw(B, H, T, seed=4).abs()
        n = len(lens) if lens else B
        s0, do, dsf = draw(n, H, Dk, Dv, seed=5), draw(B, H, T, Dv, seed=6), draw(n, H, Dk, Dv, seed=7)
        leaf = [x.clone().requires_grad_() for x in (q, k, v, g, s0)]
        o, sf = attention(*leaf, lens, 0.7)
        ro, rs = ref.linattn(q, k, v, g, s0, lens, 0.7)
        torch.testing.assert_close(o.detach(), ro, **CLOSE)
        torch.testing.assert_close(sf.detach(), rs, **CLOSE)
        want = torch.autograd.grad((o * do).sum() + (sf * dsf).sum(), leaf)
        for x, y in zip(ref.linattn_bwd(q, k, v, g, do, s0, dsf, lens, 0.7), want):
            torch.testing.assert_close(x, y, **CLOSE)


def test_gradient_of_a_decay_a_head():
    q, k, v, g = draw(2, 2, 6, 3, seed=1), draw(2, 2, 6, 3, seed=2), draw(2, 2, 6, 4, seed=3), -draw(2, seed=4).abs()
    do = draw(2, 2, 6, 4, seed=5)
    leaf = g.clone().requires_grad_()
    zero = torch.zeros(2, 2, 3, 4, dtype=torch.float64)
    o, _ = attention(q, k, v, leaf[None, :, None].expand(2, 2, 6), zero, None, 1.0)
    (want,) = torch.autograd.grad((o * do).sum(), leaf)
    torch.testing.assert_close(ref.linattn_bwd(q, k, v, g, do)[3], want, **CLOSE)


def test_steps_make_a_prompt():
    B, H, Hk, T, D = 2, 4, 2, 9, 3
    q, k, v, g = draw(B, Hk, T, D, seed=1), draw(B, Hk, T, D, seed=2), draw(B, H, T, D, seed=3), -draw(B, H, T, seed=4).abs()
    o, end = ref.linattn(q, k, v, g, scale=0.5)
    state = torch.zeros(B, H, D, D, dtype=torch.float64)
    for t in range(T):
        got, state = ref.step(q[:, :, t], k[:, :, t], v[:, :, t], g[:, :, t], state, scale=0.5)
        torch.testing.assert_close(got, o[:, :, t], **CLOSE)
    torch.testing.assert_close(state, end, **CLOSE)


def test_worked_values():
    """One key, one value: the states 1, 1/2 + 2, and the delta rule's correction."""
    one = lambda *x: torch.tensor(x, dtype=torch.float64).reshape(1, 1, -1, 1)  # noqa: E731
    g = torch.tensor([0.0, math.log(0.5)], dtype=torch.float64).reshape(1, 1, 2)
    o, s = ref.linattn(one(1, 3), one(1, 1), one(1, 2), g)
    assert o.flatten().tolist() == [1.0, 7.5] and float(s) == 2.5
    o, s = ref.step(one(2)[:, :, 0], one(1)[:, :, 0], one(5)[:, :, 0], torch.zeros(1, 1), torch.ones(1, 1, 1, 1),
                    beta=torch.tensor([[0.5]]))
    assert float(s) == 3.0 and float(o) == 6.0  # 1 + 0.5 (5 - 1)


def test_norm_and_its_gradients():
    x, w, res, dy, dres = draw(3, 7, seed=1), draw(7, seed=2), draw(3, 7, seed=3), draw(3, 7, seed=4), draw(3, 7, seed=5)
    h, y = ref.rms_norm(x, w, res)
    torch.testing.assert_close(h, x + res, **CLOSE)
    leaf = [h.clone().requires_grad_(), w.clone().requires_grad_()]
    z = leaf[0] * torch.rsqrt(leaf[0].square().mean(-1, keepdim=True) + 1e-6) * leaf[1]
    torch.testing.assert_close(z.detach(), y, **CLOSE)
    want = torch.autograd.grad((z * dy).sum(), leaf)
    dx, dw = ref.rms_norm_bwd(dy, h, w, dres)
    torch.testing.assert_close(dx, want[0] + dres, **CLOSE)
    torch.testing.assert_close(dw, want[1], **CLOSE)
