"""Timed cases of the linear-attention layer's operators: attention with a decay
for each head over packed prompts (forward and backward), its single-token step
and the gated delta rule's, the residual root-mean-square norm with 8-bit
output, and the pool of recurrent states with its forks and compactions.

Every operator has a plain form here, in elementary torch operations and 32-bit
arithmetic, next to the call of this package that computes the same.  ``own``
says which of the two ``run`` takes.  ``exact`` is the definition in 64 bits,
token by token, for the outputs that are computed numbers.
"""
import math

import torch

own = False

C = 64  # tokens per chunk of the plain chunked form
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short prompt of one user: launch latency and a ragged tail count
        dict(name="prompt 1x130", op="prompt", dtype="bf16", B=1, H=16, Hk=16, T=130, Dk=128, Dv=128, lens="",
             per_head=False, states=False),
        # the benchmark's default shape: a batch of equal prompts, no state kept
        dict(name="prompt 4x4096", op="prompt", dtype="bf16", B=4, H=16, Hk=16, T=4096, Dk=128, Dv=128, lens="",
             per_head=False, states=False),
        # a server's prefill: ragged prompts packed token-major into one row, one of them much longer, value heads
        # sharing query and key heads, states carried in and out, one request with nothing new
        dict(name="prompt packed 32760", op="prompt", dtype="bf16", B=1, H=32, Hk=16, T=32760, Dk=128, Dv=128,
             lens="17,2048,0,21001,333,4096,1,5264", per_head=False, states=True),
        # the benchmark's default shape in training
        dict(name="train 4x4096", op="train", dtype="bf16", B=4, H=16, Hk=16, T=4096, Dk=128, Dv=128, lens="",
             per_head=False, states=False),
        # ragged documents in full precision with a fixed decay a head, states and their gradients
        dict(name="train packed f32", op="train", dtype="f32", B=1, H=8, Hk=4, T=1999, Dk=64, Dv=64,
             lens="700,65,1,1233", per_head=True, states=True),
        # one user's next token
        dict(name="step 1", op="step", dtype="bf16", B=1, H=16, Hk=16, Dk=128, Dv=128, slots=4, delta=False, idle=0),
        # a full decoding batch of the gated delta rule, some of its rows idle
        dict(name="step 256 delta", op="step", dtype="bf16", B=256, H=32, Hk=16, Dk=128, Dv=128, slots=300, delta=True,
             idle=5),
        # the norm in front of a decoding batch's projections, 8-bit output
        dict(name="norm 8x2048 e4m3", op="norm", dtype="bf16", rows=8, C=2048, group=128, out="e4m3", residual=True),
        # the same over a long prompt
        dict(name="norm 32760x2048 e4m3", op="norm", dtype="bf16", rows=32760, C=2048, group=128, out="e4m3",
             residual=True),
        # the norm's backward in training, with the residual stream's gradient
        dict(name="norm back 16384x2048", op="norm_back", dtype="bf16", rows=16384, C=2048, residual=True),
        # one request forked once, and one new page
        dict(name="pool fork 2", op="fork", L=1, slots=64, H=16, Dk=128, Dv=128, n=2, live=40),
        # a pool over several layers closed up after many requests ended
        dict(name="pool compact 400", op="compact", L=6, slots=400, H=16, Dk=128, Dv=128, live=190),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, T, most):
    """Sequence lengths that add up to T: a text, empty where the row is one sequence."""
    n = rng.randint(1, max(1, min(most, T)))
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "step", "step", "norm", "norm_back", "fork", "compact"])
    if op in ("prompt", "train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Dk, Dv = (128, 128) if dtype == "bf16" and rng.random() < 0.7 else (rng.choice([64, 128]), rng.choice([64, 128]))
        Hk = _log(rng, 1, 32)
        H = Hk * rng.choice([1, 1, 2, 4])
        most = (1 << 20 if op == "prompt" else 1 << 18) // (1 if dtype == "bf16" else 8)  # tokens x heads
        packed = rng.random() < 0.5
        B = 1 if packed else _log(rng, 1, 8)
        T = min(_log(rng, 1, 32768 if op == "prompt" else 8192), max(1, most // (H * B)))
        return dict(op=op, dtype=dtype, B=B, H=H, Hk=Hk, T=T, Dk=Dk, Dv=Dv, lens=_lens(rng, T, 24) if packed else "",
                    per_head=rng.random() < 0.25, states=rng.random() < 0.5)
    if op == "step":
        B, Hk = _log(rng, 1, 256), _log(rng, 1, 16)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, H=Hk * rng.choice([1, 2]), Hk=Hk,
                    Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128]), slots=B + rng.randint(0, 40),
                    delta=rng.random() < 0.5, idle=rng.randint(0, B // 8))
    if op in ("norm", "norm_back"):
        rows, cols = _log(rng, 1, 32768), rng.choice([_log(rng, 64, 4096), 128 * rng.randint(1, 40)])
        rows = min(rows, (1 << 25) // cols)
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), rows=rows, C=cols, residual=rng.random() < 0.7)
        if op == "norm":
            case["out"] = rng.choice(["e4m3", "e4m3", "same"])
            case["group"] = 128 if case["out"] == "e4m3" and cols % 128 == 0 and rng.random() < 0.7 else 0
        return case
    slots, H = _log(rng, 8, 400), rng.randint(1, 16)
    live = rng.randint(1, slots - 2)
    case = dict(op=op, L=rng.randint(1, 6), slots=slots, H=H, Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128]), live=live)
    if op == "fork":
        case["n"] = rng.randint(1, min(slots - live + 2, 64))
    return case


# ---------------------------------------------------------------- their inputs
def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def _lengths(case):
    return [int(x) for x in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["B"]


def _chunks(case):
    """(token of each place of each chunk or -1, sequence of each chunk, last chunk of each sequence or -1): the plan
    that a program with the plain form keeps for a batch.  Tokens are counted over [B, T]."""
    at, seq, last, t0 = [], [], [], 0
    for s, n in enumerate(_lengths(case)):
        for c in range(0, n, C):
            at.append([t0 + c + j if c + j < n else -1 for j in range(C)])
            seq.append(s)
        last.append(len(at) - 1 if n else -1)
        t0 += n
    return at, seq, last


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    st = dict(case=case)
    if op in ("prompt", "train"):
        dt, B, H, Hk, T, Dk, Dv = DT[case["dtype"]], *(case[n] for n in ("B", "H", "Hk", "T", "Dk", "Dv"))
        lens = _lengths(case)
        packed = bool(case["lens"])

        def tokens(heads, width, f):  # packed prompts lie token-major, batches head-major
            x = f(randn(B, T, heads, width) if packed else randn(B, heads, T, width)).to(dt)
            return x.transpose(1, 2) if packed else x

        st["q"], st["k"], st["v"] = tokens(Hk, Dk, _unit), tokens(Hk, Dk, _unit), tokens(H, Dv, lambda x: x)
        gate = torch.nn.functional.logsigmoid(randn(H) + 2.0 if case["per_head"] else randn(B, H, T))
        st["g"] = gate if case["per_head"] else gate / 16.0
        st["s0"] = 0.3 * randn(len(lens), H, Dk, Dv) if case["states"] else None
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if packed else None
        st["n_seq"] = len(lens)
        if op == "train":
            st["do"] = tokens(H, Dv, lambda x: x)
            st["dsf"] = 0.3 * randn(len(lens), H, Dk, Dv) if case["states"] else None
        at, seq, last = _chunks(case)
        st["at"], st["seq"], st["last"] = (torch.tensor(x, device=dev) for x in (at, seq, last))
        back = torch.full((B * T,), 0, device=dev)
        flat = st["at"].reshape(-1)
        back[flat[flat >= 0]] = torch.nonzero(flat >= 0).reshape(-1)
        st["back"] = back
    elif op == "step":
        dt, B, H, Hk, Dk, Dv = DT[case["dtype"]], *(case[n] for n in ("B", "H", "Hk", "Dk", "Dv"))
        st["q"], st["k"], st["v"] = _unit(randn(B, Hk, Dk)).to(dt), _unit(randn(B, Hk, Dk)).to(dt), randn(B, H, Dv).to(dt)
        st["g"] = torch.nn.functional.logsigmoid(randn(B, H)) / 16.0
        st["beta"] = torch.sigmoid(randn(B, H)).to(dt) if case["delta"] else None
        st["state"] = randn(case["slots"], H, Dk, Dv)
        st["state_out"] = torch.zeros_like(st["state"])
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[:B].to(torch.int32)
        if case["idle"]:
            slots[torch.randperm(B, generator=gen, device=dev)[: case["idle"]]] = -1
        st["slots"] = slots
    elif op in ("norm", "norm_back"):
        dt, rows, cols = DT[case["dtype"]], case["rows"], case["C"]
        st["x"] = randn(rows, cols).to(dt)
        st["res"] = (2.0 * randn(rows, cols)).to(dt) if case["residual"] else None
        st["w"] = 1.0 + 0.1 * randn(cols)
        if op == "norm_back":
            st["dy"] = randn(rows, cols).to(dt)
    else:
        st["pool"] = randn(case["L"], case["slots"], case["H"], case["Dk"], case["Dv"])
        order = torch.randperm(case["slots"], generator=gen, device=dev)
        live = torch.zeros(case["slots"], dtype=torch.uint8, device=dev)
        live[order[: case["live"]]] = 1
        st["live"] = live
        if op == "fork":  # the last one of two or more is a new request: a page of zeros
            pick = torch.randint(case["live"], (case["n"],), generator=gen, device=dev)
            st["parents"] = order[: case["live"]][pick].to(torch.int32)
            if case["n"] > 1:
                st["parents"][-1] = -1
    return st


# ---------------------------------------------------------------- plain forms
def _segsum(x):
    """y[..., t, s] = x[s+1] + ... + x[t] for s <= t, -inf above: summed from s on, so that nothing cancels."""
    n = x.shape[-1]
    y = x[..., :, None].expand(*x.shape, n)
    low = torch.ones(n, n, dtype=torch.bool, device=x.device).tril()
    y = y.masked_fill(~low.tril(-1), 0.0).cumsum(-2)
    return y.masked_fill(~low, -math.inf)


def _plain_attention(st, q, k, v, g, s0):
    """o [B,H,T,Dv] and the final states from 32-bit q, k, v, g [B,H,T], s0, chunk by chunk."""
    B, H, T, Dv = v.shape
    at, seq, last = st["at"], st["seq"], st["last"]

    def cut(x):  # [B,h,T,...] -> [h,chunks,C,...], zeros in the places past a sequence's end
        x = x.transpose(0, 1).reshape(x.shape[1], B * T, *x.shape[3:])
        y = x[:, at.clamp_min(0)]
        return torch.where((at >= 0).reshape(1, *at.shape, *[1] * (x.dim() - 2)), y, torch.zeros((), device=x.device))

    rep = H // q.shape[1]
    q, k, v, g = cut(q).repeat_interleave(rep, 0), cut(k).repeat_interleave(rep, 0), cut(v), cut(g)
    cum = g.cumsum(-1)
    o = ((q @ k.transpose(-1, -2)) * _segsum(g).exp()) @ v
    to_end = g.flip(-1).cumsum(-1).flip(-1) - g
    U = (k * to_end.exp()[..., None]).transpose(-1, -2) @ v
    whole = cum[..., -1]
    n = len(seq)
    same = seq[:, None] == seq[None, :]
    before = torch.ones(n, n, dtype=torch.bool, device=q.device).tril(-1) & same
    # the state that enters chunk c: the earlier chunks' shares, each decayed over the chunks between
    between = _segsum(whole).roll(1, -2)  # row c: the chunks after c' and before c
    mix = torch.where(before, between, torch.full((), -math.inf, device=q.device)).exp()
    S = (mix @ U.reshape(H, n, -1)).reshape(U.shape)
    if s0 is not None:
        since = torch.where(before, whole[:, None, :], torch.zeros((), device=q.device)).sum(-1).exp()
        S = S + since[..., None, None] * s0.transpose(0, 1)[:, seq]
    o = o + cum.exp()[..., None] * (q @ S)
    out = o.reshape(H, n * C, Dv)[:, st["back"]].reshape(H, B, T, Dv).transpose(0, 1)
    end = (whole.exp()[..., None, None] * S + U).transpose(0, 1)[last.clamp_min(0)]
    kept = s0 if s0 is not None else torch.zeros_like(end)
    return out, torch.where((last >= 0)[:, None, None, None], end, kept)


def _wide(g, v):
    return g if g.dim() == 3 else g[None, :, None].expand(v.shape[0], v.shape[1], v.shape[2])


def _plain_prompt(st):
    q, k, v = (st[n].float() for n in "qkv")
    o, sf = _plain_attention(st, q, k, v, _wide(st["g"], v), st["s0"])
    return dict(o=o.to(st["v"].dtype), final_state=sf) if st["case"]["states"] else dict(o=o.to(st["v"].dtype))


def _plain_train(st):
    leaf = {n: st[n].float().detach().clone().requires_grad_() for n in ("q", "k", "v", "g", "s0") if st[n] is not None}
    o, sf = _plain_attention(st, leaf["q"], leaf["k"], leaf["v"], _wide(leaf["g"], leaf["v"]), leaf.get("s0"))
    loss = (o * st["do"].float()).sum()
    if st["dsf"] is not None:
        loss = loss + (sf * st["dsf"]).sum()
    got = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    out = {"d" + n: got[n].to(st[n].dtype) for n in ("q", "k", "v", "g")}
    if "s0" in got:
        out["ds0"] = got["s0"]
    return out


def _plain_step(st):
    case, dt = st["case"], st["v"].dtype
    busy = st["slots"] >= 0
    at = st["slots"][busy].long()
    rep = case["H"] // case["Hk"]
    q, k = (st[n].float().repeat_interleave(rep, 1)[busy] for n in "qk")
    S = st["g"][busy].exp()[..., None, None] * st["state"][at]
    u = st["v"].float()[busy]
    if case["delta"]:
        u = st["beta"].float()[busy][..., None] * (u - (k[..., None, :] @ S)[..., 0, :])
    S = S + k[..., :, None] * u[..., None, :]
    o = torch.zeros(st["v"].shape, device=S.device)
    o[busy] = (q[..., None, :] @ S)[..., 0, :]
    st["state_out"][at] = S
    return dict(o=o.to(dt), state=st["state_out"])


EPS = 1e-6
TOP = 448.0  # the largest e4m3 value


def _plain_norm(st):
    case, x = st["case"], st["x"].float()
    h = x + st["res"].float() if st["res"] is not None else x
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["w"]
    out = dict(h=h.to(st["x"].dtype)) if st["res"] is not None else {}
    if case["out"] == "same":
        return dict(out, y=y.to(st["x"].dtype))
    y = y.reshape(case["rows"], -1, case["group"] or case["C"])
    scale = (y.abs().amax(-1) / TOP).clamp_min(1e-12)
    q = (y / scale[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return dict(out, y=q.reshape(case["rows"], -1), scale=scale)


def _plain_norm_back(st):
    h, dy = st["x"].float(), st["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n, t = h * r, dy * st["w"]
    dx = r * (t - n * (n * t).mean(-1, keepdim=True))
    if st["res"] is not None:
        dx = dx + st["res"].float()
    return dict(dx=dx.to(st["x"].dtype), dw=(dy * n).sum(0))


def _plain_fork(st):
    pool, live, parents = st["pool"], st["live"].clone(), st["parents"]
    free = torch.nonzero(live == 0).reshape(-1)[: len(parents)]
    n = len(free)  # where the pool is full the rest get none
    from_, page = parents[:n].long(), (1, -1, 1, 1, 1)
    pool[:, free] = torch.where((from_ >= 0).reshape(page), pool[:, from_.clamp_min(0)], torch.zeros((), device=pool.device))
    live[free] = 1
    children = torch.full_like(parents, -1)
    children[:n] = free.to(torch.int32)
    return dict(pool=pool, live=live, children=children)


def _plain_compact(st):
    pool, live = st["pool"], st["live"]
    n, at = live.sum(dtype=torch.int32), torch.arange(len(live), device=live.device, dtype=torch.int32)
    to, from_ = torch.nonzero((live == 0) & (at < n)).reshape(-1), torch.nonzero((live == 1) & (at >= n)).reshape(-1)
    pool[:, to] = pool[:, from_]
    remap = torch.where(live == 1, at, torch.full_like(at, -1))
    remap[from_] = to.to(torch.int32)
    return dict(pool=pool, live=(at < n).to(torch.uint8), remap=remap, n=n.reshape(1))


PLAIN = dict(prompt=_plain_prompt, train=_plain_train, step=_plain_step, norm=_plain_norm, norm_back=_plain_norm_back,
             fork=_plain_fork, compact=_plain_compact)


# ---------------------------------------------------------------- this package's calls
def _own(st):
    from gated_delta_rule_47_gb300 import binding as b
    case, op = st["case"], st["case"]["op"]
    if op == "prompt":
        o, sf = b.linattn_chunk_fwd(st["q"], st["k"], st["v"], st["g"], initial_state=st["s0"], cu_seqlens=st["cu"],
                                    output_final_state=case["states"])
        return dict(o=o, final_state=sf) if case["states"] else dict(o=o)
    if op == "train":
        dq, dk, dv, dg, ds0 = b.linattn_chunk_bwd(st["q"], st["k"], st["v"], st["g"], st["do"], initial_state=st["s0"],
                                                  dfinal_state=st["dsf"], cu_seqlens=st["cu"])
        out = dict(dq=dq, dk=dk, dv=dv, dg=dg)
        return dict(out, ds0=ds0) if ds0 is not None else out
    if op == "step":
        more = dict(slots=st["slots"], state_out=st["state_out"])
        if case["delta"]:
            o = b.gdn_step(st["q"], st["k"], st["v"], st["beta"], st["g"], st["state"], **more)
        else:
            o = b.linattn_step(st["q"], st["k"], st["v"], st["g"], st["state"], **more)
        return dict(o=o, state=st["state_out"])
    if op == "norm":
        y, scale, h = b.rms_norm_fwd(st["x"], st["w"], residual=st["res"], eps=EPS, group=case["group"],
                                     out_dtype=torch.float8_e4m3fn if case["out"] == "e4m3" else None)
        out = dict(y=y) if scale is None else dict(y=y, scale=scale)
        return dict(out, h=h) if st["res"] is not None else out
    if op == "norm_back":
        dx, dw = b.rms_norm_bwd(st["dy"], st["x"], st["w"], dresidual=st["res"], eps=EPS)
        return dict(dx=dx, dw=dw)
    live = st["live"].clone()
    if op == "fork":
        children = b.state_pool_fork(st["pool"], live, st["parents"])
        return dict(pool=st["pool"], live=live, children=children)
    remap, n = b.state_pool_compact(st["pool"], live)
    return dict(pool=st["pool"], live=live, remap=remap, n=n)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("prompt", "train"):
        size, heads, Dk, Dv = (2 if case["dtype"] == "bf16" else 4), case["H"], case["Dk"], case["Dv"]
        n = case["B"] * case["T"]
        qk, v, state = 2 * n * case["Hk"] * Dk * size, n * heads * Dv * size, heads * Dk * Dv * 4 * len(_lengths(case))
        gate = heads * 4 if case["per_head"] else n * heads * 4
        state = state if case["states"] else 0
        if op == "prompt":  # one state update and one product with the state for each token
            return dict(bytes=qk + 2 * v + gate + 2 * state, flops=4 * n * heads * Dk * Dv)
        return dict(bytes=2 * qk + 3 * v + 2 * gate + 3 * state, flops=10 * n * heads * Dk * Dv)
    if op == "step":
        size, n = (2 if case["dtype"] == "bf16" else 4), case["B"] - case["idle"]
        page = case["H"] * case["Dk"] * case["Dv"]
        rows = 2 * case["Hk"] * case["Dk"] + 2 * case["H"] * case["Dv"] + (case["H"] if case["delta"] else 0)
        return dict(bytes=n * (2 * page * 4 + rows * size + case["H"] * 4), flops=n * page * (6 if case["delta"] else 4))
    if op in ("norm", "norm_back"):
        size, n = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["C"]
        if op == "norm_back":
            return dict(bytes=n * size * (4 if case["residual"] else 3) + 8 * case["C"], flops=10 * n)
        y = n if case["out"] == "e4m3" else n * size
        scales = 4 * (n // (case["group"] or case["C"])) if case["out"] == "e4m3" else 0
        return dict(bytes=n * size * (3 if case["residual"] else 1) + y + scales + 4 * case["C"], flops=6 * n)
    page = case["H"] * case["Dk"] * case["Dv"] * 4 * case["L"]
    if op == "fork":
        n = min(case["n"], case["slots"] - case["live"])
        fresh = 1 if case["n"] > 1 and n == case["n"] else 0
        return dict(bytes=page * (2 * n - fresh) + 2 * case["slots"], flops=0)
    moves = case["live"] * (case["slots"] - case["live"]) / case["slots"]  # expected
    return dict(bytes=2 * page * moves + 6 * case["slots"], flops=0)


# ---------------------------------------------------------------- the definitions in 64 bits
def _padded(case, x, fill=0.0):
    """[B,h,T,...] -> [sequences, longest, h, ...] in 64 bits, and the lengths."""
    lens = _lengths(case)
    x = x.double().transpose(1, 2).reshape(case["B"] * case["T"], x.shape[1], *x.shape[3:])
    out = torch.full((len(lens), max(lens), *x.shape[1:]), fill, dtype=torch.float64, device=x.device)
    t = 0
    for s, n in enumerate(lens):
        out[s, :n] = x[t: t + n]
        t += n
    return out


def _unpadded(case, x, like):
    rows = torch.cat([x[s, :n] for s, n in enumerate(_lengths(case))])
    return rows.reshape(case["B"], case["T"], *x.shape[2:]).transpose(1, 2).reshape(like.shape)


def _exact_prompt(case, st):
    rep = case["H"] // case["Hk"]
    q, k, v = (_padded(case, st[n]) for n in "qkv")
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    decay = _padded(case, _wide(st["g"], st["v"])).exp()  # 1 past a sequence's end, where k is 0: the state stays
    S = torch.zeros(q.shape[0], case["H"], case["Dk"], case["Dv"], dtype=torch.float64, device=q.device)
    if st["s0"] is not None:
        S += st["s0"].double()
    o = torch.empty_like(v)
    for t in range(q.shape[1]):
        S.mul_(decay[:, t, :, None, None]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
        o[:, t] = (q[:, t, :, None, :] @ S)[..., 0, :]
    o = _unpadded(case, o, st["v"])
    return dict(o=o, final_state=S) if case["states"] else dict(o=o)


def _exact_train(case, st):
    rep = case["H"] // case["Hk"]
    q, k, v, do = (_padded(case, st[n]) for n in ("q", "k", "v", "do"))
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    decay = _padded(case, _wide(st["g"], st["v"])).exp()
    n, L = q.shape[:2]
    S = torch.zeros(n, case["H"], case["Dk"], case["Dv"], dtype=torch.float64, device=q.device)
    R = torch.zeros_like(S)
    if st["s0"] is not None:
        S += st["s0"].double()
    if st["dsf"] is not None:
        R += st["dsf"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S.mul_(decay[:, t, :, None, None]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
        dq[:, t] = (S @ do[:, t, :, :, None])[..., 0]
    ends = (R * S).sum((-1, -2))  # the last decay's share that comes from the final state
    for t in range(L - 1, -1, -1):
        R.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :])
        dk[:, t], dv[:, t] = (R @ v[:, t, :, :, None])[..., 0], (k[:, t, :, None, :] @ R)[..., 0, :]
        R.mul_(decay[:, t, :, None, None])
    dg = ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(1).cumsum(1).flip(1) + ends[:, None]
    shared = lambda x: x.reshape(n, L, case["Hk"], rep, -1).sum(3)  # noqa: E731
    out = dict(dq=_unpadded(case, shared(dq), st["q"]), dk=_unpadded(case, shared(dk), st["k"]),
               dv=_unpadded(case, dv, st["v"]))
    dg = _unpadded(case, dg[..., None], st["v"][..., :1])[..., 0]
    out["dg"] = dg.sum((0, 2)) if case["per_head"] else dg
    return dict(out, ds0=R) if st["s0"] is not None else out


def _exact_step(case, st):
    B, H, rep = case["B"], case["H"], case["H"] // case["Hk"]
    o = torch.zeros(B, H, case["Dv"], dtype=torch.float64, device="cuda")
    state = torch.zeros(st["state"].shape, dtype=torch.float64, device="cuda")
    for b, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        q, k = (st[n][b].double().repeat_interleave(rep, 0) for n in "qk")
        S = st["state"][slot].double() * st["g"][b].double().exp()[:, None, None]
        u = st["v"][b].double()
        if case["delta"]:
            u = st["beta"][b].double()[:, None] * (u - torch.einsum("hi,hij->hj", k, S))
        S = S + torch.einsum("hi,hj->hij", k, u)
        o[b], state[slot] = torch.einsum("hi,hij->hj", q, S), S
    return dict(o=o, state=state)


def _exact_norm(case, st):
    h = st["x"].double()
    h = h + st["res"].double() if st["res"] is not None else h
    y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["C"] + EPS) * st["w"].double()
    out = dict(h=h) if st["res"] is not None else {}
    if case["out"] == "same":
        return dict(out, y=y)
    y = y.reshape(case["rows"], -1, case["group"] or case["C"])
    scale = (y.abs().max(-1).values / TOP).clamp_min(1e-12)
    return dict(out, y=(y / scale[..., None]).reshape(case["rows"], -1), scale=scale)


def _exact_norm_back(case, st):
    h, dy, w = st["x"].double(), st["dy"].double(), st["w"].double()
    m = (h * h).sum(-1, keepdim=True) / case["C"] + EPS
    dx = dy * w / m.sqrt() - h * (dy * w * h).sum(-1, keepdim=True) / (case["C"] * m ** 1.5)
    if st["res"] is not None:
        dx = dx + st["res"].double()
    return dict(dx=dx, dw=(dy * h / m.sqrt()).sum(0))


def exact(case, seed):
    by = dict(prompt=_exact_prompt, train=_exact_train, step=_exact_step, norm=_exact_norm, norm_back=_exact_norm_back)
    if case["op"] not in by:  # pages are moved, not computed
        return None
    return by[case["op"]](case, prepare(case, seed))
