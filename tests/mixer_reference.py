"""Plain 64-bit forms of the operators next to a mixer, token by token and on the
CPU, for the tests of the CUDA kernels.  Gradients are those that torch derives
from them."""
from __future__ import annotations

import torch


def sequences(B, T, cu=None):
    """(row, first token, end) of every sequence; offsets outside the row are cut to it."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cut = [min(max(int(c), 0), T) for c in cu]
    return [(0, a, max(a, b)) for a, b in zip(cut, cut[1:])]


def wide(t):
    return None if t is None else t.detach().double().cpu()


def silu(x):
    return x / (1 + torch.exp(-x))


def conv(x, w, bias=None, win=None, cu=None, act=True):
    """y [B,T,C] and the windows that sequences leave; tokens of no sequence give 0."""
    B, T, C = x.shape
    W = w.shape[1]
    y, wins = torch.zeros(B, T, C, dtype=torch.float64), []
    rows = []
    for s, (b, t0, t1) in enumerate(sequences(B, T, cu)):
        past = torch.zeros(W - 1, C, dtype=torch.float64) if win is None else win[s]
        seq = torch.cat([past, x[b, t0:t1]])
        rows += [(b, t, (seq[t - t0: t - t0 + W] * w.t()).sum(0)) for t in range(t0, t1)]
        wins.append(seq[len(seq) - (W - 1):])
    for b, t, z in rows:
        z = z if bias is None else z + bias
        y = y.index_put((torch.tensor(b), torch.tensor(t)), silu(z) if act else z)
    return y, torch.stack(wins)


def scan(x, dt, A, B, C, D=None, z=None, bias=None, s0=None, cu=None, soft=True):
    """y [B,T,Di] and the final states; tokens of no sequence give 0."""
    rows, T, Di = x.shape
    v = dt if bias is None else dt + bias
    step = torch.logaddexp(v, torch.zeros_like(v)) if soft else v
    outs, states = {}, []
    for s, (b, t0, t1) in enumerate(sequences(rows, T, cu)):
        h = torch.zeros(Di, A.shape[1], dtype=torch.float64) if s0 is None else s0[s]
        for t in range(t0, t1):
            h = torch.exp(step[b, t][:, None] * A) * h + (step[b, t] * x[b, t])[:, None] * B[b, t]
            o = (h * C[b, t]).sum(-1)
            if D is not None:
                o = o + D * x[b, t]
            outs[b, t] = o if z is None else o * silu(z[b, t])
        states.append(h)
    none = torch.zeros(Di, dtype=torch.float64)
    y = torch.stack([torch.stack([outs.get((b, t), none) for t in range(T)]) for b in range(rows)]) if rows * T else x
    return y, torch.stack(states)


def gated(x, g, w=None, eps=1e-6, first=False, sigmoid=False):
    act = 1 / (1 + torch.exp(-g))
    act = act if sigmoid else g * act
    u = x * act if first else x
    y = u / ((u * u).mean(-1, keepdim=True) + eps).sqrt()
    y = y if w is None else y * w
    return y if first else y * act


def block(x, res, w1=None, s=None, w2=None, eps=1e-6):
    """y and h of rows [n,C]."""
    norm = lambda u, w: u / ((u * u).mean(-1, keepdim=True) + eps).sqrt() * (1 if w is None else w)  # noqa: E731
    n = norm(x, w1)
    if s is not None:
        s = s.reshape(-1, x.shape[-1])
        n = n * s.repeat_interleave(len(x) // len(s), 0)
    h = res + n
    return norm(h, w2), h


def leaves(**tensors):
    """64-bit copies, their gradients wanted."""
    return {n: None if t is None else wide(t).requires_grad_() for n, t in tensors.items()}


def grads(outs, couts, inputs):
    """Gradients of sum(out * cout) by each input; None stays."""
    loss = sum((o * c).sum() for o, c in zip(outs, couts) if c is not None)
    given = {n: t for n, t in inputs.items() if t is not None}
    if not torch.is_tensor(loss) or not loss.requires_grad:  # no token reaches anything
        return {n: None if t is None else torch.zeros_like(t) for n, t in inputs.items()}
    got = torch.autograd.grad(loss, list(given.values()), allow_unused=True)
    full = {n: torch.zeros_like(t) if g is None else g for (n, t), g in zip(given.items(), got)}
    return {n: full.get(n) for n in inputs}
