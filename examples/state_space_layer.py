"""A state space layer served and trained with the library's operators.

The layer: norm -> projection -> short convolution -> selective scan with its gate
-> output projection -> norm after the block, its scale, the residual's sum and the
norm before the next block.  Serving keeps each request's window and state in one
page each of two pools: prompts of different lengths go through one packed call,
then every request takes one token a step.  Training runs the same layer forwards
and backwards.

    python examples/state_space_layer.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gated_delta_rule_47_gb300 import binding  # noqa: E402


class Layer:
    """Weights of one layer of width C with Di channels of N states and W taps."""

    def __init__(self, C=256, Di=512, N=16, W=4, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen).to(device)  # noqa: E731
        proj = lambda a, b: (randn(a, b) / a ** 0.5).bfloat16()  # noqa: E731
        self.C, self.Di, self.N, self.W = C, Di, N, W
        self.win, self.wdbc, self.wout = proj(C, 2 * Di), proj(Di, Di + 2 * N), proj(Di, C)
        self.taps, self.bias = randn(Di, W) / W ** 0.5, torch.zeros(Di, device=device)
        self.A = -torch.arange(1, N + 1, device=device).float().expand(Di, N).contiguous()
        self.D, self.dt_bias = torch.ones(Di, device=device), torch.full((Di,), -4.0, device=device)
        self.pre, self.post, self.next = (torch.ones(C, device=device) for _ in range(3))
        self.scale = torch.full((C,), 0.5, device=device)

    def inner(self, y, conv, scan):
        """The block between the norms on normed rows y [..,C]; conv and scan keep what they carry."""
        xz = y @ self.win
        x = conv(xz[..., :self.Di])
        dbc = x @ self.wdbc
        dt, B, C = dbc.split([self.Di, self.N, self.N], -1)
        return scan(x, dt, B, C, xz[..., self.Di:]) @ self.wout

    def prefill(self, x, residual, lengths, windows, states, pages):
        """Packed prompts x, residual [tokens,C]; what they carry goes to `pages` of both pools.  Returns the next
        block's input and its residual."""
        cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=x.device)

        def conv(x):
            y, windows[pages.long()] = binding.causal_conv_fwd(x, self.taps, self.bias, output_final_window=True, cu_seqlens=cu)
            return y

        def scan(x, dt, B, C, z):
            y, states[pages.long()] = binding.ssm_scan_fwd(x, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias,
                                                           output_final_state=True, cu_seqlens=cu)
            return y
        y, _, h = binding.rms_norm_fwd(x[None], self.pre, residual=residual[None])
        y, h = binding.block_norm_fwd(self.inner(y, conv, scan), h, self.post, self.scale, self.next)
        return y[0], h[0]

    def decode(self, x, residual, windows, states, slots):
        """One token of each request: x, residual [requests,C], slots int32 (-1: idle)."""
        y, _, h = binding.rms_norm_fwd(x, self.pre, residual=residual)
        o = self.inner(y, lambda x: binding.causal_conv_step(x, self.taps, windows, self.bias, slots=slots),
                       lambda x, dt, B, C, z: binding.ssm_step(x, dt, self.A, B, C, states, D=self.D, z=z, dt_bias=self.dt_bias,
                                                               slots=slots))
        return binding.block_norm_fwd(o, h, self.post, self.scale, self.next)

    def train_step(self, x, residual, target):
        """Loss and gradients by name for rows x, residual, target [B,T,C]."""
        kept = {}

        def conv(x):
            kept["x"] = x
            return binding.causal_conv_fwd(x, self.taps, self.bias)[0]

        def scan(*args):
            kept["args"] = args
            x, dt, B, C, z = args
            kept["y"] = binding.ssm_scan_fwd(x, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias)[0]
            return kept["y"]
        u, _, h0 = binding.rms_norm_fwd(x, self.pre, residual=residual)
        o = self.inner(u, conv, scan)
        y, h = binding.block_norm_fwd(o, h0, self.post, self.scale, self.next)
        loss = (y.float() - target).square().mean()
        dy = ((y.float() - target) * (2 / y.numel())).bfloat16()
        g = {}
        do, dh, g["post"], g["scale"], g["next"] = binding.block_norm_bwd(dy, None, o, h, self.post, self.scale, self.next)
        xs, dt, B, C, z = kept["args"]
        dxs, ddt, g["A"], dB, dC, g["D"], dz, g["dt_bias"], _ = binding.ssm_scan_bwd(
            xs, dt, self.A, B, C, do @ self.wout.t(), D=self.D, z=z, dt_bias=self.dt_bias)
        ddbc = torch.cat([ddt, dB, dC], -1)
        dxc, g["taps"], g["bias"], _ = binding.causal_conv_bwd(kept["x"], self.taps, dxs + ddbc @ self.wdbc.t(), self.bias)
        dxz = torch.cat([dxc, dz], -1)
        for name, a, b in (("wout", kept["y"], do), ("wdbc", xs, ddbc), ("win", u, dxz)):
            g[name] = a.flatten(0, -2).t() @ b.flatten(0, -2)
        g["x"], g["pre"] = binding.rms_norm_bwd(dxz @ self.win.t(), h0, self.pre, dresidual=dh)
        return float(loss), g


def serve(layer, lengths=(37, 130, 5), slots=8, steps=3, seed=1):
    """Prefill, then steps; returns each call's output rows."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda n: torch.randn(n, layer.C, generator=gen).cuda().bfloat16()  # noqa: E731
    windows = torch.zeros(slots, layer.W - 1, layer.Di, device="cuda", dtype=torch.bfloat16)
    states = torch.zeros(slots, layer.Di, layer.N, device="cuda")
    pages = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    outs = [layer.prefill(rand(sum(lengths)), rand(sum(lengths)), list(lengths), windows, states, pages)[0]]
    for _ in range(steps):
        outs.append(layer.decode(rand(len(lengths)), rand(len(lengths)), windows, states, pages)[0])
    return outs


def main():
    layer = Layer()
    outs = serve(layer)
    print(f"served: prompts {tuple(outs[0].shape)}, {len(outs) - 1} steps of {len(outs[1])} requests")
    x, res = (torch.randn(2, 150, layer.C, device="cuda").bfloat16() for _ in range(2))
    loss, g = layer.train_step(x, res, torch.randn(2, 150, layer.C, device="cuda"))
    print(f"trained: loss {loss:.4f}, " + ", ".join(f"|d{n}| {float(t.float().norm()):.2e}" for n, t in g.items()))


if __name__ == "__main__":
    main()
