"""Plain 64-bit forms of the operators around a linear-attention layer, token
by token and on the CPU, for the tests of the CUDA kernels."""
from __future__ import annotations

import torch


def sequences(B, T, lens):
    """(row, first token, tokens) of every sequence; lens None: one a row."""
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    out, t = [], 0
    for n in lens:
        out.append((0, t, n))
        t += n
    return out


def linattn(q, k, v, g, s0=None, lens=None, scale=1.0, first=0):
    """o [B,H,T,Dv] and the final states; lens: lengths packed from token
    `first` on; tokens of no sequence give 0.  g [B,H,T] or [H]."""
    q, k, v, g = (x.double().cpu() for x in (q, k, v, g))
    B, H, T, Dv = v.shape
    rep = H // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    if g.dim() == 1:
        g = g[None, :, None].expand(B, H, T)
    o, states = torch.zeros(B, H, T, Dv, dtype=torch.float64), []
    for s, (row, t0, n) in enumerate(sequences(B, T, lens)):
        t0 += first
        S = torch.zeros(H, q.shape[-1], Dv, dtype=torch.float64) if s0 is None else s0[s].double().cpu().clone()
        for t in range(t0, t0 + n):
            S = g[row, :, t].exp()[:, None, None] * S + k[row, :, t, :, None] * v[row, :, t, None, :]
            o[row, :, t] = scale * (q[row, :, t, None, :] @ S)[:, 0]
        states.append(S)
    return o, torch.stack(states)


def linattn_bwd(q, k, v, g, do, s0=None, dsf=None, lens=None, scale=1.0, first=0):
    """dq, dk, dv, dg, ds0 by the recurrences of the state and of its gradient."""
    per_head, Hk = g.dim() == 1, q.shape[1]
    q, k, v, g, do = (x.double().cpu() for x in (q, k, v, g, do))
    B, H, T, Dv = v.shape
    rep, Dk = H // Hk, q.shape[-1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    if per_head:
        g = g[None, :, None].expand(B, H, T)
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros(B, H, T, dtype=torch.float64)
    ds0 = []
    for s, (row, t0, n) in enumerate(sequences(B, T, lens)):
        t0 += first
        S = [torch.zeros(H, Dk, Dv, dtype=torch.float64) if s0 is None else s0[s].double().cpu()]
        for t in range(t0, t0 + n):
            S.append(g[row, :, t].exp()[:, None, None] * S[-1] + k[row, :, t, :, None] * v[row, :, t, None, :])
        R = torch.zeros(H, Dk, Dv, dtype=torch.float64) if dsf is None else dsf[s].double().cpu().clone()
        for t in reversed(range(t0, t0 + n)):
            R = R + scale * q[row, :, t, :, None] * do[row, :, t, None, :]
            dq[row, :, t] = scale * (S[t - t0 + 1] @ do[row, :, t, :, None])[..., 0]
            dk[row, :, t] = (R @ v[row, :, t, :, None])[..., 0]
            dv[row, :, t] = (k[row, :, t, None, :] @ R)[:, 0]
            e = g[row, :, t].exp()
            dg[row, :, t] = e * (R * S[t - t0]).sum((-1, -2))
            R = e[:, None, None] * R
        ds0.append(R)
    dq, dk = (x.reshape(B, Hk, rep, T, Dk).sum(2) for x in (dq, dk))
    return dq, dk, dv, dg.sum((0, 2)) if per_head else dg, torch.stack(ds0)


def step(q, k, v, g, state, slots=None, beta=None, scale=1.0, l2norm=False):
    """o [B,H,Dv] and the states after one token; slots out of range are idle."""
    q, k, v, g, state = (x.double().cpu() for x in (q, k, v, g, state))
    B, H, Dv = v.shape
    rep = H // q.shape[1]
    if l2norm:
        q, k = (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12) for x in (q, k))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    if g.dim() == 1:
        g = g[None].expand(B, H)
    o, state = torch.zeros(B, H, Dv, dtype=torch.float64), state.clone()
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < state.shape[0]:
            continue
        D = g[b].exp()[:, None, None] * state[s]
        u = v[b]
        if beta is not None:
            u = beta[b].double().cpu()[:, None] * (u - (k[b][:, None, :] @ D)[:, 0])
        state[s] = D + k[b][:, :, None] * u[:, None, :]
        o[b] = scale * (q[b][:, None, :] @ state[s])[:, 0]
    return o, state


def rms_norm(x, w=None, res=None, eps=1e-6):
    """h and y, unrounded."""
    h = x.double().cpu()
    if res is not None:
        h = h + res.double().cpu()
    y = h / ((h * h).mean(-1, keepdim=True) + eps).sqrt()
    return h, y if w is None else y * w.double().cpu()


def rms_norm_bwd(dy, h, w=None, dres=None, eps=1e-6):
    dy, h = dy.double().cpu(), h.double().cpu()
    C = h.shape[-1]
    m = (h * h).mean(-1, keepdim=True) + eps
    t = dy if w is None else dy * w.double().cpu()
    dx = t / m.sqrt() - h * (t * h).sum(-1, keepdim=True) / (C * m ** 1.5)
    if dres is not None:
        dx = dx + dres.double().cpu()
    return dx, (dy * h / m.sqrt()).reshape(-1, C).sum(0)
