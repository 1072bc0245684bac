"""A linear-attention layer served and trained with the library's operators.

The layer: residual RMS norm -> projections -> linear attention with a decay for
each head (or, decoding, the gated delta rule) -> output projection.  Serving
keeps each request's state in one page of a pool: prompts of different lengths
go through one packed call, then every request takes one token a step; requests
fork, end, and the pool is closed up.  Training runs the same layer forwards and
backwards.

    python examples/linear_attention_layer.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gated_delta_rule_47_gb300 import binding  # noqa: E402


class Layer:
    """Weights of one layer of width C with H value heads on Hk query / key heads of D."""

    def __init__(self, C=512, H=4, Hk=2, D=128, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=gen) / s[0] ** 0.5).to(device)  # noqa: E731
        self.C, self.H, self.Hk, self.D, self.scale = C, H, Hk, D, D ** -0.5
        self.norm = torch.ones(C, device=device)
        self.wqkv = rand(C, (2 * Hk + H) * D).bfloat16()
        self.wgate = rand(C, 2 * H).bfloat16()
        self.wout = rand(H * D, C).bfloat16()

    def project(self, y):
        """q, k [n,Hk,D], v [n,H,D], log-decay [n,H], beta [n,H] of normed rows."""
        n, H, Hk, D = y.shape[0], self.H, self.Hk, self.D
        qkv = (y @ self.wqkv).view(n, 2 * Hk + H, D)
        gates = (y @ self.wgate).float().view(n, 2, H)
        q, k, v = qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).bfloat16()  # noqa: E731
        return unit(q), unit(k), v.contiguous(), torch.nn.functional.logsigmoid(gates[:, 0] + 2), torch.sigmoid(gates[:, 1]).bfloat16()

    def normed(self, x, residual):
        """The norm's 8-bit output with its scales, as a bf16 operand; and the new residual."""
        y, scales, h = binding.rms_norm_fwd(x, self.norm, residual=residual, out_dtype=torch.float8_e4m3fn, group=128)
        y = (y.float().view(len(x), -1, 128) * scales[..., None]).view_as(x).bfloat16()
        return y, h

    def prefill(self, x, residual, lengths, pool, pages):
        """Packed prompts x, residual [tokens,C]; their states go to `pages` of pool [1,slots,H,D,D]."""
        y, h = self.normed(x, residual)
        q, k, v, g, _ = self.project(y)
        cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=x.device)
        row = lambda t: t.unsqueeze(0).transpose(1, 2)  # noqa: E731  [n,heads,D] -> [1,heads,n,D]
        o, states = binding.linattn_chunk_fwd(row(q), row(k), row(v), row(g), cu_seqlens=cu, scale=self.scale,
                                              output_final_state=True)
        pool[0, pages.long()] = states
        return o.squeeze(0).transpose(0, 1).reshape(len(x), -1) @ self.wout, h

    def decode(self, x, residual, pool, slots, delta=False):
        """One token of each request: x, residual [requests,C], slots int32 (-1: idle)."""
        y, h = self.normed(x, residual)
        q, k, v, g, beta = self.project(y)
        if delta:
            o = binding.gdn_step(q, k, v, beta, g, pool[0], slots=slots, scale=self.scale)
        else:
            o = binding.linattn_step(q, k, v, g, pool[0], slots=slots, scale=self.scale)
        return o.reshape(len(x), -1) @ self.wout, h

    def train_step(self, x, target):
        """Loss and the gradients of the attention's inputs and of the norm for rows x [T,C]."""
        y, _, h = binding.rms_norm_fwd(x, self.norm)
        y = y.detach().requires_grad_()
        q, k, v, g, _ = self.project(y)
        row = lambda t: t.detach().unsqueeze(0).transpose(1, 2)  # noqa: E731
        args = row(q), row(k), row(v), row(g)
        o, _ = binding.linattn_chunk_fwd(*args, scale=self.scale)
        rows = o.squeeze(0).transpose(0, 1).reshape(len(x), -1).detach().requires_grad_()
        loss = ((rows @ self.wout).float() - target).square().mean()
        (dout,) = torch.autograd.grad(loss, rows)
        dout = dout.view(len(x), self.H, self.D).unsqueeze(0).transpose(1, 2)
        dq, dk, dv, dg, _ = binding.linattn_chunk_bwd(*args, dout, scale=self.scale)
        back = lambda t: t.squeeze(0).transpose(0, 1)  # noqa: E731
        (dy,) = torch.autograd.grad((q, k, v, g), y, (back(dq), back(dk), back(dv), back(dg)))
        dx, dnorm = binding.rms_norm_bwd(dy.contiguous(), h, self.norm)
        return float(loss.detach()), dx, dnorm


def serve(layer, lengths=(37, 130, 5), slots=8, steps=3, seed=1):
    """Prefill, decode, fork, end and compact; returns each request's outputs."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda n: torch.randn(n, layer.C, generator=gen).cuda().bfloat16()  # noqa: E731
    pool = torch.zeros(1, slots, layer.H, layer.D, layer.D, device="cuda")
    live = torch.zeros(slots, dtype=torch.uint8, device="cuda")
    pages = binding.state_pool_fork(pool, live, torch.full((len(lengths),), -1, dtype=torch.int32, device="cuda"))
    n = sum(lengths)
    prompt, _ = layer.prefill(rand(n), rand(n), list(lengths), pool, pages)
    outs = [prompt]
    # the second request goes on in two ways
    child = binding.state_pool_fork(pool, live, pages[1:2])
    requests = torch.cat([pages, child])
    for _ in range(steps):
        o, _ = layer.decode(rand(len(requests)), rand(len(requests)), pool, requests)
        outs.append(o)
    # the first request ends; the others' pages close up
    binding.state_pool_free(live, requests[:1])
    remap, n_live = binding.state_pool_compact(pool, live)
    requests = remap[requests[1:].long()]
    o, _ = layer.decode(rand(len(requests)), rand(len(requests)), pool, requests)
    outs.append(o)
    return outs, requests, int(n_live)


def main():
    layer = Layer()
    outs, requests, n_live = serve(layer)
    print(f"served: prompts {tuple(outs[0].shape)}, {len(outs) - 1} steps, {n_live} requests live in slots {requests.tolist()}")
    x, target = torch.randn(300, layer.C, device="cuda").bfloat16(), torch.randn(300, layer.C, device="cuda")
    loss, dx, dnorm = layer.train_step(x, target)
    print(f"trained: loss {loss:.4f}, |dx| {float(dx.float().norm()):.3e}, |dnorm| {float(dnorm.norm()):.3e}")


if __name__ == "__main__":
    main()
