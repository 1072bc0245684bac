"""Timed cases of the operators next to a recurrent layer's mixer: the short
causal convolution in front of it (prompts, training, single tokens), the
selective state space scan with a decay for each channel and state (prompts,
training, single tokens), the norm by head with a gate behind it, and the norms
after a block and before the next with the scaled residual between.

Every operator has a plain form here, in elementary torch operations and 32-bit
arithmetic, next to the call of this package that computes the same.  ``own``
says which of the two ``run`` takes.  ``exact`` is the definition in 64 bits,
token by token where the operator has a recurrence.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    packs = "17,2048,0,21001,333,4096,1,5264"
    return [
        # a server's prefill: the convolution of 16 query, 16 key and 32 value heads over ragged prompts packed into one
        # row, one of them much longer, windows carried in and out, one request with nothing new
        dict(name="conv prompt packed 32760", op="conv", dtype="bf16", B=1, T=32760, C=8192, W=4, lens=packs, bias=False,
             silu=True, states=True),
        # the same in front of 16 heads of query, key and value in training, a batch of equal rows
        dict(name="conv train 4x4096", op="conv_back", dtype="bf16", B=4, T=4096, C=6144, W=4, lens="", bias=True, silu=True,
             states=False),
        # a full decoding batch, some of its rows idle
        dict(name="conv step 256", op="conv_step", dtype="bf16", B=256, C=8192, W=4, slots=300, idle=5, bias=False, silu=True),
        # one short prompt of one user
        dict(name="scan prompt 1x130", op="scan", dtype="bf16", B=1, T=130, Di=2048, N=16, lens="", gate=True, skip=True,
             states=False),
        # the packed prefill's scan, states carried in and out
        dict(name="scan prompt packed 32760", op="scan", dtype="bf16", B=1, T=32760, Di=2048, N=16, lens=packs, gate=True,
             skip=True, states=True),
        # a batch in training
        dict(name="scan train 4x4096", op="scan_back", dtype="bf16", B=4, T=4096, Di=2048, N=16, lens="", gate=True, skip=True,
             states=False),
        # ragged documents in full precision, states and their gradients
        dict(name="scan train packed f32", op="scan_back", dtype="f32", B=1, T=1999, Di=512, N=16, lens="700,65,1,1233",
             gate=False, skip=True, states=True),
        # a full decoding batch
        dict(name="scan step 256", op="scan_step", dtype="bf16", B=256, Di=2048, N=16, slots=300, idle=5, gate=True, skip=True),
        # eight users' next tokens: the norm of 16 heads in front of the output projection
        dict(name="gated norm 8x16x128", op="gated", dtype="bf16", B=1, T=8, H=16, D=128, shared=True, gate_first=False,
             sigmoid=False, heads_first=False),
        # its gradients in training, at the layout that the attention's heads come in
        dict(name="gated norm back 4x4096x16x128", op="gated_back", dtype="bf16", B=4, T=4096, H=16, D=128, shared=True,
             gate_first=False, sigmoid=False, heads_first=True),
        # between two blocks of a decoding batch
        dict(name="block norm 8x2048", op="block", dtype="bf16", rows=8, C=2048, groups=1),
        # between two blocks in training, with the residual stream's gradient
        dict(name="block norm back 16384x2048", op="block_back", dtype="bf16", rows=16384, C=2048, groups=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, T, most):
    """Sequence lengths that add up to T: a text."""
    n = rng.randint(1, max(1, min(most, T)))
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["conv", "conv_back", "conv_step", "scan", "scan", "scan_back", "scan_back", "scan_step", "gated",
                     "gated_back", "block", "block_back"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    coin = lambda p: rng.random() < p  # noqa: E731
    narrow = 1 if dtype == "bf16" else 2
    if op in ("conv", "conv_back", "scan", "scan_back"):
        conv = op.startswith("conv")
        most = {"conv": 1 << 28, "conv_back": 96 << 20, "scan": 64 << 20, "scan_back": 32 << 20}[op] // narrow
        wide = 8 * _log(rng, 1, 1024 if conv else 512)
        packed = coin(0.5)
        B = 1 if packed else _log(rng, 1, 8)
        T = min(_log(rng, 1, 32768 if not op.endswith("back") else 8192), max(1, most // (wide * B)))
        case = dict(op=op, dtype=dtype, B=B, T=T, lens=_lens(rng, T, 24) if packed else "", states=coin(0.5))
        if conv:
            return dict(case, C=wide, W=rng.choice([2, 3, 4, 4]), bias=coin(0.5), silu=coin(0.8))
        N = rng.choice([8, 16, 16, 16, 32])
        case["T"] = T = min(T, max(1, most * 16 // (wide * B * N)))
        if packed:
            case["lens"] = _lens(rng, T, 24)
        return dict(case, Di=wide, N=N, gate=coin(0.7), skip=coin(0.8))
    if op in ("conv_step", "scan_step"):
        B = _log(rng, 1, 256)
        case = dict(op=op, dtype=dtype, B=B, slots=B + rng.randint(0, 40), idle=rng.randint(0, B // 8))
        if op == "conv_step":
            return dict(case, C=8 * _log(rng, 1, 1024), W=rng.choice([2, 3, 4, 4]), bias=coin(0.5), silu=coin(0.8))
        return dict(case, Di=8 * _log(rng, 1, 256), N=rng.choice([8, 16, 16, 32]), gate=coin(0.7), skip=coin(0.8))
    if op in ("gated", "gated_back"):
        H, D = _log(rng, 1, 32), rng.choice([64, 128, 128, 256, 8 * rng.randint(1, 256)])
        B = _log(rng, 1, 8)
        T = min(_log(rng, 1, 16384), max(1, (1 << 25) // narrow // (B * H * D)))
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, D=D, shared=coin(0.6), gate_first=coin(0.3), sigmoid=coin(0.3),
                    heads_first=coin(0.4))
    C = rng.choice([8 * _log(rng, 8, 512), 128 * rng.randint(1, 40)])
    groups = rng.choice([0, 1, 1, rng.randint(2, 8)])
    each = max(1, groups)
    rows = each * max(1, min(_log(rng, 1, 32768), (1 << 25) // narrow // C) // each)
    return dict(op=op, dtype=dtype, rows=rows, C=C, groups=groups)


# ---------------------------------------------------------------- their inputs
def _lengths(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["B"]


def _plan(case, st):
    """Where the sequences lie in the B*T tokens: the plan that a program keeps for a batch."""
    lens, dev = _lengths(case), "cuda"
    first = [0]
    for n in lens:
        first.append(first[-1] + n)
    pos = torch.cat([torch.arange(n) for n in lens]).to(dev)
    left = torch.cat([torch.arange(n - 1, -1, -1) for n in lens]).to(dev)
    st["cu"] = torch.tensor(first, dtype=torch.int32, device=dev) if case["lens"] else None
    st.update(first=torch.tensor(first[:-1], device=dev), len=torch.tensor(lens, device=dev), pos=pos, left=left)
    st["some"] = torch.tensor([i for i, n in enumerate(lens) if n], dtype=torch.long, device=dev)
    st["n_seq"] = len(lens)


def prepare(case, seed):
    dev, op, dt = "cuda", case["op"], DT[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    st = dict(case=case)
    if "slots" in case:
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[: case["B"]].to(torch.int32)
        if case["idle"]:
            slots[torch.randperm(case["B"], generator=gen, device=dev)[: case["idle"]]] = -1
        st["slots"] = slots
    elif "lens" in case:
        _plan(case, st)
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        rows = (case["B"], C) if op == "conv_step" else (case["B"], case["T"], C)
        st["x"] = randn(*rows).to(dt)
        st["w"] = randn(C, W) / W ** 0.5
        st["b"] = 0.1 * randn(C) if case["bias"] else None
        if op == "conv_step":
            st["window"] = randn(case["slots"], W - 1, C).to(dt)
            st["window_out"] = torch.zeros_like(st["window"])
        else:
            st["win"] = randn(st["n_seq"], W - 1, C).to(dt) if case["states"] else None
        if op == "conv_back":
            st["dy"] = randn(*rows).to(dt)
            st["dwin"] = randn(st["n_seq"], W - 1, C).to(dt) if case["states"] else None
    elif op.startswith("scan"):
        Di, N = case["Di"], case["N"]
        rows = (case["B"],) if op == "scan_step" else (case["B"], case["T"])
        st["x"] = torch.nn.functional.silu(randn(*rows, Di)).to(dt)
        st["dt"] = (0.5 * randn(*rows, Di)).to(dt)
        step = torch.exp(math.log(1e-3) + rand(Di) * math.log(1e2))  # steps of 0.001 to 0.1 where dt is 0
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["A"] = -torch.arange(1, N + 1, device=dev) * torch.exp(0.1 * randn(Di, N))
        st["B"], st["C"] = randn(*rows, N).to(dt), randn(*rows, N).to(dt)
        st["D"] = 1.0 + 0.1 * randn(Di) if case["skip"] else None
        st["z"] = randn(*rows, Di).to(dt) if case["gate"] else None
        if op == "scan_step":
            st["state"] = randn(case["slots"], Di, N)
            st["state_out"] = torch.zeros_like(st["state"])
        else:
            st["s0"] = 0.3 * randn(st["n_seq"], Di, N) if case["states"] else None
        if op == "scan_back":
            st["dy"] = randn(*rows, Di).to(dt)
            st["dsf"] = 0.3 * randn(st["n_seq"], Di, N) if case["states"] else None
    elif op.startswith("gated"):
        B, T, H, D = (case[n] for n in ("B", "T", "H", "D"))
        x = randn(B, H, T, D) if case["heads_first"] else randn(B, T, H, D)
        st["x"] = x.to(dt).transpose(1, 2) if case["heads_first"] else x.to(dt)
        st["g"] = randn(B, T, H, D).to(dt)
        st["w"] = 1.0 + 0.1 * (randn(D) if case["shared"] else randn(H, D))
        if op == "gated_back":
            st["dy"] = randn(B, T, H, D).to(dt)
    else:
        rows, C = case["rows"], case["C"]
        st["x"], st["res"] = randn(rows, C).to(dt), (2.0 * randn(rows, C)).to(dt)
        st["w1"], st["w2"] = 1.0 + 0.1 * randn(C), 1.0 + 0.1 * randn(C)
        st["s"] = 0.5 + 0.1 * randn(case["groups"], C) if case["groups"] else None
        if op == "block_back":
            x = st["x"].float()
            s = st["s"].repeat_interleave(rows // case["groups"], 0) if case["groups"] else 1.0
            st["h"] = (st["res"].float() + s * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w1"]).to(dt)
            st["dy"], st["dh"] = randn(rows, C).to(dt), randn(rows, C).to(dt)
    return st


# ---------------------------------------------------------------- plain forms
def _silu_back(z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def _before(st, x, n, win, W):
    """x[t - n] of every token [n_tokens,C], from the window (or 0) before a sequence's start."""
    if n == 0:
        return x
    y = torch.zeros_like(x)
    y[n:] = x[: max(len(x) - n, 0)]
    y = torch.where((st["pos"] >= n)[:, None], y, torch.zeros((), device=x.device))
    if win is not None:
        for p in range(n):
            on = st["len"] > p
            y[(st["first"] + p)[on]] = win[on, W - 1 + p - n]
    return y


def _conv(st, x, win):
    W = st["w"].shape[1]
    z = sum(_before(st, x, W - 1 - j, win, W) * st["w"][:, j] for j in range(W))
    return z if st["b"] is None else z + st["b"]


def _window(st, x, win, W):
    """The last W - 1 inputs of every sequence, counted over its window and its tokens."""
    out = torch.zeros(st["n_seq"], W - 1, x.shape[-1], dtype=x.dtype, device=x.device)
    for r in range(W - 1):
        at = st["len"] + r
        if win is not None:
            out[:, r] = win[torch.arange(st["n_seq"], device=x.device), at.clamp_max(W - 2)]
        own_ = at >= W - 1
        out[own_, r] = x[(st["first"] + at - (W - 1))[own_]]
    return out


def _plain_conv(st):
    case, x = st["case"], st["x"].float().flatten(0, 1)
    win = None if st["win"] is None else st["win"].float()
    z = _conv(st, x, win)
    y = (z * torch.sigmoid(z) if case["silu"] else z).to(st["x"].dtype).reshape(st["x"].shape)
    return dict(y=y, window=_window(st, x, win, case["W"]).to(st["x"].dtype)) if case["states"] else dict(y=y)


def _plain_conv_back(st):
    case, x, dy = st["case"], st["x"].float().flatten(0, 1), st["dy"].float().flatten(0, 1)
    W, dt, w = case["W"], st["x"].dtype, st["w"]
    win = None if st["win"] is None else st["win"].float()
    dz = dy * _silu_back(_conv(st, x, win)) if case["silu"] else dy
    dx, dw, dwin = torch.zeros_like(x), torch.zeros_like(w), None if win is None else torch.zeros_like(win)
    for n in range(W):
        dw[:, W - 1 - n] = (dz * _before(st, x, n, win, W)).sum(0)
        later = torch.zeros_like(dz)
        later[: max(len(dz) - n, 0)] = dz[n:]
        dx += torch.where((st["left"] >= n)[:, None], later, torch.zeros((), device=x.device)) * w[:, W - 1 - n]
    if win is not None:
        for r in range(W - 1):
            for p in range(r + 1):  # token p of a sequence reaches window row r by tap r - p
                on = st["len"] > p
                dwin[on, r] += dz[(st["first"] + p)[on]] * w[:, r - p]
            at = st["len"] + r
            own_, d = at >= W - 1, st["dwin"][:, r].float()
            dx[(st["first"] + at - (W - 1))[own_]] += d[own_]
            dwin[~own_, at[~own_]] += d[~own_]
    out = dict(dx=dx.to(dt).reshape(st["x"].shape), dw=dw)
    if st["b"] is not None:
        out["db"] = dz.sum(0)
    return dict(out, dwindow=dwin.to(dt)) if win is not None else out


def _plain_conv_step(st):
    case = st["case"]
    busy = st["slots"] >= 0
    at = st["slots"][busy].long()
    rows = torch.cat([st["window"][at], st["x"][busy][:, None]], 1)
    z = (rows.float() * st["w"].t()).sum(1)
    if st["b"] is not None:
        z = z + st["b"]
    y = torch.zeros(st["x"].shape, device=z.device)
    y[busy] = z * torch.sigmoid(z) if case["silu"] else z
    st["window_out"][at] = rows[:, 1:]
    return dict(y=y.to(st["x"].dtype), window=st["window_out"])


def _softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


def _doubled(a, b):
    """h[t] = a[t] h[t-1] + b[t] over the first axis: both are overwritten, b is the answer."""
    n = 1
    while n < len(a):
        b[n:] += a[n:] * b[:-n]  # the product is whole before anything is written
        a[n:] *= a[:-n].clone()
        n *= 2
    return b


def _scan_parts(st):
    """Tokens as one axis: x, steps, decays [n,Di,N], inputs of the state, each in 32 bits."""
    x = st["x"].float().flatten(0, 1)
    v = st["dt"].float().flatten(0, 1) + st["dt_bias"]
    step = _softplus(v)
    a = torch.exp(step[..., None] * st["A"])
    u = (step * x)[..., None] * st["B"].float().flatten(0, 1)[:, None]
    return x, v, step, a, u


def _states(st, a, u):
    """h of every token, from the decays and the state's inputs (overwritten)."""
    on = st["some"]
    if st["s0"] is not None:
        u[st["first"][on]] += a[st["first"][on]] * st["s0"][on]
    a = a.clone()
    a[st["first"][on]] = 0
    return _doubled(a, u)


def _plain_scan(st):
    case = st["case"]
    x, _, _, a, u = _scan_parts(st)
    h = _states(st, a, u)
    y = (h * st["C"].float().flatten(0, 1)[:, None]).sum(-1)
    if st["D"] is not None:
        y = y + st["D"] * x
    if st["z"] is not None:
        z = st["z"].float().flatten(0, 1)
        y = y * z * torch.sigmoid(z)
    out = dict(y=y.to(st["x"].dtype).reshape(st["x"].shape))
    if case["states"]:
        last = st["s0"].clone()
        on = st["some"]
        last[on] = h[(st["first"] + st["len"] - 1)[on]]
        out["state"] = last
    return out


def _plain_scan_back(st):
    dt, on, shape = st["x"].dtype, st["some"], st["x"].shape
    B, C, dy = (st[n].float().flatten(0, 1) for n in ("B", "C", "dy"))
    x, v, step, a, u = _scan_parts(st)
    h = _states(st, a, u)
    out = {}
    if st["z"] is not None:
        z = st["z"].float().flatten(0, 1)
        y = (h * C[:, None]).sum(-1)
        if st["D"] is not None:
            y = y + st["D"] * x
        out["dz"] = (dy * y * _silu_back(z)).to(dt).reshape(shape)
        dy = dy * z * torch.sigmoid(z)
    out["dC"] = (h * dy[..., None]).sum(1).to(dt).reshape(st["C"].shape)
    # g[t] = C[t] dy[t] + a[t+1] g[t+1]: the same recurrence from the end
    first, last = st["first"][on], (st["first"] + st["len"] - 1)[on]
    g = C[:, None] * dy[..., None]
    if st["dsf"] is not None:
        g[last] += st["dsf"][on]
    after = torch.zeros_like(a)
    after[:-1] = a[1:]
    after[last] = 0
    g = _doubled(after.flip(0), g.flip(0)).flip(0)
    del after
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    del h
    prev[first] = st["s0"][on] if st["s0"] is not None else 0
    if st["s0"] is not None:
        out["dstate"] = st["dsf"].clone()
        out["dstate"][on] = a[first] * g[first]
    prev *= a
    prev *= g  # what passes over each decay's exponent
    out["dA"] = (prev * step[..., None]).sum(0)
    gB = (g * B[:, None]).sum(-1)
    dstep = (prev * st["A"]).sum(-1) + x * gB
    dv = dstep * torch.sigmoid(v)
    dx = step * gB
    if st["D"] is not None:
        dx = dx + st["D"] * dy
        out["dD"] = (dy * x).sum(0)
    out["dB"] = (g * (step * x)[..., None]).sum(1).to(dt).reshape(st["B"].shape)
    return dict(out, dx=dx.to(dt).reshape(shape), ddt=dv.to(dt).reshape(shape), ddt_bias=dv.sum(0))


def _plain_scan_step(st):
    busy = st["slots"] >= 0
    at = st["slots"][busy].long()
    x, B, C = (st[n][busy].float() for n in ("x", "B", "C"))
    step = _softplus(st["dt"][busy].float() + st["dt_bias"])
    h = torch.exp(step[..., None] * st["A"]) * st["state"][at] + (step * x)[..., None] * B[:, None]
    v = (h * C[:, None]).sum(-1)
    if st["D"] is not None:
        v = v + st["D"] * x
    if st["z"] is not None:
        z = st["z"][busy].float()
        v = v * z * torch.sigmoid(z)
    y = torch.zeros(st["x"].shape, device=x.device)
    y[busy] = v
    st["state_out"][at] = h
    return dict(y=y.to(st["x"].dtype), state=st["state_out"])


def _act(case, g):
    s = torch.sigmoid(g)
    return s if case["sigmoid"] else g * s


def _plain_gated(st):
    case, x, a = st["case"], st["x"].float(), _act(st["case"], st["g"].float())
    if case["gate_first"]:
        x = x * a
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w"]
    return dict(y=(y if case["gate_first"] else y * a).to(st["x"].dtype))


def _plain_gated_back(st):
    case, dt = st["case"], st["x"].dtype
    x, g, dy = st["x"].float(), st["g"].float(), st["dy"].float()
    s = torch.sigmoid(g)
    act, slope = (s, s * (1 - s)) if case["sigmoid"] else (g * s, _silu_back(g))
    u = x * act if case["gate_first"] else x
    r = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    n = u * r
    t = dy if case["gate_first"] else dy * act  # the gradient of w n
    tw = t * st["w"]
    du = r * (tw - n * (n * tw).mean(-1, keepdim=True))
    dg = du * x * slope if case["gate_first"] else dy * n * st["w"] * slope
    dx = du * act if case["gate_first"] else du
    return dict(dx=dx.to(dt), dgate=dg.to(dt), dw=(t * n).sum((0, 1, 2) if case["shared"] else (0, 1)))


def _scale_rows(st):
    case = st["case"]
    return st["s"].repeat_interleave(case["rows"] // case["groups"], 0) if case["groups"] else 1.0


def _plain_block(st):
    x = st["x"].float()
    h = st["res"].float() + _scale_rows(st) * (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w1"])
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["w2"]
    return dict(y=y.to(st["x"].dtype), h=h.to(st["x"].dtype))


def _plain_block_back(st):
    case, dt = st["case"], st["x"].dtype
    x, h, dy, s = st["x"].float(), st["h"].float(), st["dy"].float(), _scale_rows(st)
    r2 = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n2, t2 = h * r2, dy * st["w2"]
    dres = st["dh"].float() + r2 * (t2 - n2 * (n2 * t2).mean(-1, keepdim=True))
    r1 = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n1, t1 = x * r1, dres * s * st["w1"]
    dx = r1 * (t1 - n1 * (n1 * t1).mean(-1, keepdim=True))
    out = dict(dx=dx.to(dt), dres=dres.to(dt), dw1=(dres * s * n1).sum(0), dw2=(dy * n2).sum(0))
    if case["groups"]:
        out["ds"] = (dres * st["w1"] * n1).reshape(case["groups"], -1, case["C"]).sum(1)
    return out


PLAIN = dict(conv=_plain_conv, conv_back=_plain_conv_back, conv_step=_plain_conv_step, scan=_plain_scan,
             scan_back=_plain_scan_back, scan_step=_plain_scan_step, gated=_plain_gated, gated_back=_plain_gated_back,
             block=_plain_block, block_back=_plain_block_back)


# ---------------------------------------------------------------- this package's calls
def _own(st):
    from gated_delta_rule_47_gb300 import binding as b
    case, op = st["case"], st["case"]["op"]
    if op == "conv":
        y, win = b.causal_conv_fwd(st["x"], st["w"], st["b"], initial_window=st["win"], output_final_window=case["states"],
                                   cu_seqlens=st["cu"], silu=case["silu"])
        return dict(y=y, window=win) if case["states"] else dict(y=y)
    if op == "conv_back":
        dx, dw, db, dwin = b.causal_conv_bwd(st["x"], st["w"], st["dy"], st["b"], initial_window=st["win"],
                                             dfinal_window=st["dwin"], cu_seqlens=st["cu"], silu=case["silu"])
        out = dict(dx=dx, dw=dw)
        if db is not None:
            out["db"] = db
        return dict(out, dwindow=dwin) if dwin is not None else out
    if op == "conv_step":
        y = b.causal_conv_step(st["x"], st["w"], st["window"], st["b"], slots=st["slots"], window_out=st["window_out"],
                               silu=case["silu"])
        return dict(y=y, window=st["window_out"])
    if op.startswith("scan"):
        args = tuple(st[n] for n in ("x", "dt", "A", "B", "C"))
        more = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"])
    if op == "scan":
        y, state = b.ssm_scan_fwd(*args, **more, initial_state=st["s0"], output_final_state=case["states"],
                                  cu_seqlens=st["cu"])
        return dict(y=y, state=state) if case["states"] else dict(y=y)
    if op == "scan_back":
        dx, ddt, dA, dB, dC, dD, dz, dbias, ds0 = b.ssm_scan_bwd(*args, st["dy"], **more, initial_state=st["s0"],
                                                                 dfinal_state=st["dsf"], cu_seqlens=st["cu"])
        out = dict(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, dz=dz, ddt_bias=dbias, dstate=ds0)
        return {n: t for n, t in out.items() if t is not None}
    if op == "scan_step":
        return dict(y=b.ssm_step(*args, st["state"], **more, slots=st["slots"], state_out=st["state_out"]),
                    state=st["state_out"])
    if op == "gated":
        return dict(y=b.gated_norm_fwd(st["x"], st["g"], st["w"], eps=EPS, gate_first=case["gate_first"],
                                       sigmoid=case["sigmoid"]))
    if op == "gated_back":
        dx, dg, dw = b.gated_norm_bwd(st["dy"], st["x"], st["g"], st["w"], eps=EPS, gate_first=case["gate_first"],
                                      sigmoid=case["sigmoid"])
        return dict(dx=dx, dgate=dg, dw=dw)
    if op == "block":
        y, h = b.block_norm_fwd(st["x"], st["res"], st["w1"], st["s"], st["w2"], eps=EPS)
        return dict(y=y, h=h)
    dx, dres, dw1, ds, dw2 = b.block_norm_bwd(st["dy"], st["dh"], st["x"], st["h"], st["w1"], st["s"], st["w2"], eps=EPS)
    out = dict(dx=dx, dres=dres, dw1=dw1, dw2=dw2)
    return dict(out, ds=ds) if ds is not None else out


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("conv", "conv_back"):
        n, C, W = case["B"] * case["T"], case["C"], case["W"]
        windows = (W - 1) * C * size * len(_lengths(case)) if case["states"] else 0
        small = 4 * C * (W + (1 if case["bias"] else 0))
        if op == "conv":
            return dict(bytes=2 * n * C * size + 2 * windows + small, flops=(2 * W + 4) * n * C)
        return dict(bytes=3 * n * C * size + 3 * windows + 2 * small, flops=(6 * W + 10) * n * C)
    if op == "conv_step":
        n, C, W = case["B"] - case["idle"], case["C"], case["W"]
        return dict(bytes=n * C * size * 2 * W + 4 * C * W, flops=(2 * W + 4) * n * C)
    if op.startswith("scan"):
        Di, N = case["Di"], case["N"]
        gate = 1 if case["gate"] else 0
        if op == "scan_step":
            n = case["B"] - case["idle"]
            return dict(bytes=n * (Di * N * 8 + (3 + gate) * Di * size + 2 * N * size) + 4 * Di * (N + 2), flops=8 * n * Di * N)
        n = case["B"] * case["T"]
        state = Di * N * 4 * len(_lengths(case)) if case["states"] else 0
        if op == "scan":  # a decay's exponential, its argument, and three products with the state a (token, channel, state)
            return dict(bytes=n * size * ((3 + gate) * Di + 2 * N) + 2 * state + 4 * Di * (N + 2), flops=8 * n * Di * N)
        return dict(bytes=n * size * ((5 + 2 * gate) * Di + 4 * N) + 3 * state + 8 * Di * (N + 2), flops=22 * n * Di * N)
    if op.startswith("gated"):
        n, w = case["B"] * case["T"] * case["H"] * case["D"], 4 * case["D"] * (1 if case["shared"] else case["H"])
        return dict(bytes=n * size * 3 + w, flops=10 * n) if op == "gated" else dict(bytes=n * size * 5 + 2 * w, flops=24 * n)
    n, C = case["rows"] * case["C"], case["C"]
    small = 4 * C * (2 + case["groups"])
    return dict(bytes=n * size * 4 + small, flops=12 * n) if op == "block" else dict(bytes=n * size * 6 + 2 * small, flops=26 * n)


# ---------------------------------------------------------------- the definitions in 64 bits
def _sequences(case):
    """(first token, tokens) over the B*T tokens."""
    out, t = [], 0
    for n in _lengths(case):
        out.append((t, n))
        t += n
    return out


def _exact_conv(case, st):
    x, w, W, C = st["x"].double().flatten(0, 1), st["w"].double(), case["W"], case["C"]
    y, wins = torch.zeros_like(x), []
    for s, (t, n) in enumerate(_sequences(case)):
        head = st["win"][s].double() if case["states"] else torch.zeros(W - 1, C, dtype=torch.float64, device=x.device)
        rows = torch.cat([head, x[t: t + n]])
        if n:
            y[t: t + n] = (rows.unfold(0, W, 1) * w).sum(-1)
        wins.append(rows[n:])
    if st["b"] is not None:
        y = y + st["b"].double()
    if case["silu"]:
        y = y / (1 + torch.exp(-y))
    out = dict(y=y.reshape(st["x"].shape))
    return dict(out, window=torch.stack(wins)) if case["states"] else out


def _exact_conv_back(case, st):
    x, dy, w, W, C = st["x"].double().flatten(0, 1), st["dy"].double().flatten(0, 1), st["w"].double(), case["W"], case["C"]
    bias = 0 if st["b"] is None else st["b"].double()
    dx, dw, db, dwins = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(C, dtype=torch.float64, device=x.device), []
    for s, (t, n) in enumerate(_sequences(case)):
        head = st["win"][s].double() if case["states"] else torch.zeros(W - 1, C, dtype=torch.float64, device=x.device)
        rows = torch.cat([head, x[t: t + n]])
        drows = torch.zeros_like(rows)
        if case["states"]:
            drows[n:] += st["dwin"][s].double()
        if n:
            taps = rows.unfold(0, W, 1)  # [n,C,W]
            z = (taps * w).sum(-1) + bias
            e = torch.exp(-z)
            dz = dy[t: t + n] * (((1 + e) + z * e) / (1 + e) ** 2) if case["silu"] else dy[t: t + n]
            dw += (dz[..., None] * taps).sum(0)
            db += dz.sum(0)
            for j in range(W):
                drows[j: j + n] += dz * w[:, j]
        dx[t: t + n] = drows[W - 1:]
        dwins.append(drows[: W - 1])
    out = dict(dx=dx.reshape(st["x"].shape), dw=dw)
    if st["b"] is not None:
        out["db"] = db
    return dict(out, dwindow=torch.stack(dwins)) if case["states"] else out


def _exact_conv_step(case, st):
    y, wins = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda"), torch.zeros(st["window"].shape, device="cuda").double()
    for b, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        rows = torch.cat([st["window"][slot], st["x"][b: b + 1]]).double()
        z = torch.einsum("jc,cj->c", rows, st["w"].double())
        z = z if st["b"] is None else z + st["b"].double()
        y[b] = z / (1 + torch.exp(-z)) if case["silu"] else z
        wins[slot] = rows[1:]
    return dict(y=y, window=wins)


def _by_sequence(case, x):
    """[B,T,...] -> [longest, sequences, ...] in 64 bits, zeros past a sequence's end."""
    x, seqs = x.double().flatten(0, 1), _sequences(case)
    out = torch.zeros(max(n for _, n in seqs), len(seqs), *x.shape[1:], dtype=torch.float64, device=x.device)
    for s, (t, n) in enumerate(seqs):
        out[:n, s] = x[t: t + n]
    return out


def _by_token(case, x, shape):
    return torch.cat([x[:n, s] for s, (_, n) in enumerate(_sequences(case))]).reshape(shape)


def _exact_steps(case, st):
    """Steps by sequence, 0 past an end, where the state then stays; and the argument of their softplus."""
    v = _by_sequence(case, st["dt"]) + st["dt_bias"].double()
    n = torch.tensor(_lengths(case), device=v.device)
    there = torch.arange(len(v), device=v.device)[:, None] < n
    return torch.where(there[..., None], torch.log(1 + torch.exp(v)), torch.zeros((), device=v.device)), v


def _exact_scan(case, st):
    x, B, C = (_by_sequence(case, st[n]) for n in ("x", "B", "C"))
    step, _ = _exact_steps(case, st)
    A = st["A"].double()
    h = torch.zeros(x.shape[1], case["Di"], case["N"], dtype=torch.float64, device=x.device)
    if st["s0"] is not None:
        h += st["s0"].double()
    y = torch.empty_like(x)
    for t in range(len(x)):
        h.mul_(torch.exp(step[t][..., None] * A)).addcmul_((step[t] * x[t])[..., None], B[t][:, None])
        y[t] = (h @ C[t][..., None])[..., 0]
    if st["D"] is not None:
        y = y + st["D"].double() * x
    if st["z"] is not None:
        z = _by_sequence(case, st["z"])
        y = y * z / (1 + torch.exp(-z))
    out = dict(y=_by_token(case, y, st["x"].shape))
    return dict(out, state=h) if case["states"] else out


def _exact_scan_back(case, st):
    x, B, C, dy = (_by_sequence(case, st[n]) for n in ("x", "B", "C", "dy"))
    step, v = _exact_steps(case, st)
    A = st["A"].double()
    S = torch.zeros(len(x) + 1, x.shape[1], case["Di"], case["N"], dtype=torch.float64, device=x.device)
    if st["s0"] is not None:
        S[0] = st["s0"].double()
    y = torch.zeros_like(x)
    for t in range(len(x)):
        S[t + 1] = S[t] * torch.exp(step[t][..., None] * A) + (step[t] * x[t])[..., None] * B[t][:, None]
        y[t] = (S[t + 1] @ C[t][..., None])[..., 0]
    out = {}
    skip = st["D"].double() if st["D"] is not None else None
    if st["z"] is not None:
        z = _by_sequence(case, st["z"])
        e = torch.exp(-z)
        full = y if skip is None else y + skip * x
        out["dz"] = _by_token(case, dy * full * ((1 + e) + z * e) / (1 + e) ** 2, st["x"].shape)
        dy = dy * z / (1 + e)
    R = torch.zeros_like(S[0])
    if st["dsf"] is not None:
        R = R + st["dsf"].double()
    dx, dv, dB, dC, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A)
    for t in range(len(x) - 1, -1, -1):
        R = R + dy[t][..., None] * C[t][:, None]
        dC[t] = torch.einsum("sd,sdn->sn", dy[t], S[t + 1])
        dB[t] = torch.einsum("sd,sdn->sn", step[t] * x[t], R)
        RB = (R @ B[t][..., None])[..., 0]
        dx[t] = step[t] * RB
        R = R * torch.exp(step[t][..., None] * A)
        over = R * S[t]
        dv[t] = x[t] * RB + (over * A).sum(-1)
        dA += (over * step[t][..., None]).sum(0)
    dv = dv / (1 + torch.exp(-v))
    if skip is not None:
        dx = dx + skip * dy
        out["dD"] = _by_token(case, dy * x, (-1, case["Di"])).sum(0)
    if st["s0"] is not None:
        out["dstate"] = R
    dv = _by_token(case, dv, st["x"].shape)
    return dict(out, dx=_by_token(case, dx, st["x"].shape), ddt=dv, ddt_bias=dv.sum((0, 1)), dA=dA,
                dB=_by_token(case, dB, st["B"].shape), dC=_by_token(case, dC, st["C"].shape))


def _exact_scan_step(case, st):
    y, state = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(st["state"], dtype=torch.float64)
    for b, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        x, B, C = (st[n][b].double() for n in ("x", "B", "C"))
        step = torch.log(1 + torch.exp(st["dt"][b].double() + st["dt_bias"].double()))
        h = torch.exp(step[:, None] * st["A"].double()) * st["state"][slot].double() + torch.outer(step * x, B)
        y[b] = h @ C
        if st["D"] is not None:
            y[b] += st["D"].double() * x
        if st["z"] is not None:
            z = st["z"][b].double()
            y[b] *= z / (1 + torch.exp(-z))
        state[slot] = h
    return dict(y=y, state=state)


def _exact_act(case, g):
    s = 1 / (1 + torch.exp(-g))
    return (s, s - s * s) if case["sigmoid"] else (g * s, s + g * s - g * s * s)


def _norm64(x, n):
    """1 / sqrt(mean x^2 + eps) of the last axis, of n elements."""
    return 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / n + EPS)


def _back64(t, x, n):
    """The gradient of x where x _norm64(x) has the gradient t."""
    r = _norm64(x, n)
    return t * r - x * (t * x).sum(-1, keepdim=True) * r ** 3 / n


def _exact_gated(case, st):
    x, w = st["x"].double(), st["w"].double()
    act, _ = _exact_act(case, st["g"].double())
    if case["gate_first"]:
        return dict(y=x * act * _norm64(x * act, case["D"]) * w)
    return dict(y=x * _norm64(x, case["D"]) * w * act)


def _exact_gated_back(case, st):
    x, w, dy, D = st["x"].double(), st["w"].double(), st["dy"].double(), case["D"]
    act, slope = _exact_act(case, st["g"].double())
    over = (0, 1, 2) if case["shared"] else (0, 1)
    if case["gate_first"]:
        u = x * act
        du = _back64(dy * w, u, D)
        return dict(dx=du * act, dgate=du * x * slope, dw=(dy * u * _norm64(u, D)).sum(over))
    n = x * _norm64(x, D)
    return dict(dx=_back64(dy * w * act, x, D), dgate=dy * w * n * slope, dw=(dy * act * n).sum(over))


def _exact_block(case, st):
    x, C = st["x"].double(), case["C"]
    n = x * _norm64(x, C) * st["w1"].double()
    if case["groups"]:
        n = (n.reshape(case["groups"], -1, C) * st["s"].double()[:, None]).reshape(-1, C)
    h = st["res"].double() + n
    return dict(y=h * _norm64(h, C) * st["w2"].double(), h=h)


def _exact_block_back(case, st):
    x, h, dy, C = st["x"].double(), st["h"].double(), st["dy"].double(), case["C"]
    w1, w2 = st["w1"].double(), st["w2"].double()
    dres = st["dh"].double() + _back64(dy * w2, h, C)
    n, t = x * _norm64(x, C), dres
    out = dict(dres=dres, dw2=(dy * h * _norm64(h, C)).sum(0))
    if case["groups"]:
        out["ds"] = (dres * n * w1).reshape(case["groups"], -1, C).sum(1)
        t = (dres.reshape(case["groups"], -1, C) * st["s"].double()[:, None]).reshape(-1, C)
    return dict(out, dx=_back64(t * w1, x, C), dw1=(t * n).sum(0))


EXACT = dict(conv=_exact_conv, conv_back=_exact_conv_back, conv_step=_exact_conv_step, scan=_exact_scan,
             scan_back=_exact_scan_back, scan_step=_exact_scan_step, gated=_exact_gated, gated_back=_exact_gated_back,
             block=_exact_block, block_back=_exact_block_back)


def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))
