"""How the operators next to a mixer are called: inside a captured graph, twice at once
on two streams, through the long way in as through the short one, with a workspace
and outputs of the caller's, on sizes that pass 32 bits."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_causal_conv import inputs as conv_inputs
from tests.test_gpu_gated_norm import heads, rows
from tests.test_gpu_ssm_scan import backward, forward, inputs as scan_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def conv_both(d, cu=None, **kw):
    y, win = binding.causal_conv_fwd(d["x"], d["w"], d["b"], initial_window=d["win"], output_final_window=True, cu_seqlens=cu, **kw)
    return (y, win, *binding.causal_conv_bwd(d["x"], d["w"], d["dy"], d["b"], initial_window=d["win"], dfinal_window=d["dwin"],
                                             cu_seqlens=cu, **kw))


def scan_both(d, cu=None, **kw):
    return (*forward(d, cu, **kw), *backward(d, cu, **kw).values())


def norms(g, d, **kw):
    y, h = binding.block_norm_fwd(d["x"], d["res"], d["w1"], d["s"], d["w2"], **kw)
    return (binding.gated_norm_fwd(g["x"], g["g"], g["w"], **kw), *binding.gated_norm_bwd(g["dy"], g["x"], g["g"], g["w"], **kw), y, h,
            *binding.block_norm_bwd(d["dy"], d["dh"], d["x"], h, d["w1"], d["s"], d["w2"], **kw))


def calls():
    c = conv_inputs(1, 300, 64, 4, "bf16", 1, n_seq=2)
    s = scan_inputs(1, 300, 64, 16, "bf16", 2, n_seq=2)
    g, b = heads(1, 50, 4, 64, "bf16", 3, True), rows(50, 256, "bf16", 4, 1)
    cu = torch.tensor([0, 111, 300], dtype=torch.int32, device="cuda")
    return (c["x"], s["x"], g["x"], b["x"]), lambda **kw: (*conv_both(c, cu, **kw), *scan_both(s, cu, **kw), *norms(g, b, **kw))


def test_graph_replays():
    """Three replays on new inputs give what the calls give, gradients of one graph beside an eager call of the same leaves."""
    xs, call = calls()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        for x in xs:
            x.copy_(torch.randn_like(x))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert binding.device_error() == 0


def test_steps_in_a_graph():
    """Windows and states updated in place by each replay."""
    c, s = conv_inputs(4, 1, 64, 4, "bf16", 1), scan_inputs(4, 1, 64, 16, "bf16", 2)
    slots = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device="cuda")
    windows, states = torch.randn(6, 3, 64, device="cuda").bfloat16(), torch.randn(6, 64, 16, device="cuda")
    x = c["x"][:, 0].contiguous()

    def step(windows, states):
        y = binding.causal_conv_step(x, c["w"], windows, c["b"], slots=slots)
        return y, binding.ssm_step(y, s["dt"][:, 0], s["A"], s["B"][:, 0], s["C"][:, 0], states, D=s["D"], z=s["z"][:, 0],
                                   dt_bias=s["bias"], slots=slots)
    captured, called = (windows.clone(), states.clone()), (windows.clone(), states.clone())
    step(windows.clone(), states.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*captured)
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        graph.replay()
        want = step(*called)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*outs, *captured), (*want, *called)))


def test_two_streams_at_once():
    xs, call = calls()
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for s in streams:
            outs.append(call(stream=s))
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_long_way_in(monkeypatch):
    """Without the front the binding gives the same."""
    _, call = calls()
    want = call()

    class No:
        def __getattr__(self, name):
            return lambda *a: NotImplemented
    monkeypatch.setattr(binding, "_front", No())
    got = call()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_caller_workspaces():
    s = scan_inputs(2, 100, 64, 16, "f32", 2)
    need = binding._bytes("ssm_scan_bwd_workspace_bytes", 2, 100, 64, 16, binding.GDN_F32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN in every word
    a, b = backward(s), backward(s, workspace=ws)
    assert all(torch.equal(a[n], b[n]) for n in a)
    need = binding._bytes("ssm_scan_fwd_workspace_bytes", 2, 100, 64, 16, binding.GDN_F32)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(forward(s), forward(s, workspace=ws)))
    c = conv_inputs(2, 100, 64, 4, "f32", 2)
    ws = torch.full((binding._bytes("causal_conv_bwd_workspace_bytes", 2, 100, 64, 4),), 255, dtype=torch.uint8, device="cuda")
    a = binding.causal_conv_bwd(c["x"], c["w"], c["dy"], c["b"])
    b = binding.causal_conv_bwd(c["x"], c["w"], c["dy"], c["b"], workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_many_chunks_and_what_a_workspace_held():
    """Packed sequences over more chunks than are joined in place, ends at chunks' ends among them, in a workspace full
    of NaN: shares that no sequence carries on are never read."""
    for cu in ([0, 256, 4000, 4001, 9000], [700, 1024, 2048, 8000, 8500], [0, 9000, 9000, 9000, 9000]):
        s = scan_inputs(1, 9000, 16, 16, "f32", 2, n_seq=4)
        offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for f, name in ((forward, "ssm_scan_fwd_workspace_bytes"), (backward, "ssm_scan_bwd_workspace_bytes")):
            ws = torch.full((binding._bytes(name, 1, 9000, 16, 16, binding.GDN_F32),), 255, dtype=torch.uint8, device="cuda")
            a, b = f(s, offsets), f(s, offsets, workspace=ws)
            a, b = (list(t.values()) if isinstance(t, dict) else t for t in (a, b))
            assert all(torch.equal(p, q) and bool(p.isfinite().all()) for p, q in zip(a, b))
            # each sequence by itself
            if f is forward:
                for i, (t0, t1) in enumerate(zip(cu, cu[1:])):
                    one = {n: t[:, t0:t1] if n in ("x", "dt", "B", "C", "z") else t for n, t in s.items()}
                    y, last = forward(dict(one, s0=s["s0"][i: i + 1]))
                    assert float((y - a[0][:, t0:t1]).abs().max() if t1 > t0 else 0) <= 9000 * 2.0 ** -22 * float(a[0].abs().max())
                    assert float((last[0] - a[1][i]).abs().max()) <= 9000 * 2.0 ** -22 * float(a[1].abs().max())


@pytest.mark.parametrize("T,Di", [(130, 256), (700, 2048)])
def test_calls_feed_one_another(T, Di):
    """Each call reads what the one before it wrote, in the same workspace and without a wait of the host in between: a
    call's kernels, which begin while the one before ends, wait for what they read."""
    def walk(wait):
        s = scan_inputs(1, T, Di, 16, "f32", 4)
        kept = []
        for _ in range(12):
            y, last = forward(s)
            if wait:
                torch.cuda.synchronize()
            s = dict(s, x=y, s0=last)
            got = backward(s)
            if wait:
                torch.cuda.synchronize()
            s = dict(s, x=y / y.abs().amax(), dy=got["x"] / got["x"].abs().amax().clamp_min(1e-30))
            kept += [y, last, *got.values()]
        torch.cuda.synchronize()
        return kept
    for a, b in zip(walk(True), walk(False)):
        assert torch.equal(a, b)


def test_many_sequences():
    """Thousands of short and empty sequences in one row."""
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 4, (5000,), generator=gen)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    T = int(cu[-1])
    s = scan_inputs(1, T, 16, 8, "f32", 2, n_seq=5000)
    y, last = forward(s, cu.to(torch.int32).cuda())
    got = backward(s, cu.to(torch.int32).cuda())
    c = conv_inputs(1, T, 16, 4, "f32", 2, n_seq=5000)
    yc, win, dx, dw, db, dwin = conv_both(c, cu.to(torch.int32).cuda())
    # each sequence by itself, as a padded batch: steps of 0 keep the state
    at = (cu[:-1, None] + torch.arange(3)).clamp_max(T - 1).cuda()
    there = (torch.arange(3) < lens[:, None]).cuda()
    soft = lambda t: torch.nn.functional.softplus(t.float())  # noqa: E731
    batch = {n: s[n][0][at] for n in ("x", "B", "C", "z", "dy")}
    batch["dt"] = torch.where(there[..., None], s["dt"][0][at], torch.full((), -1e30, device="cuda"))
    p = dict(s, **batch)
    py, plast = forward(p)
    assert torch.equal(py[there], y[0]) and torch.equal(plast, last)
    assert bool(soft(batch["dt"]).isfinite().all())
    p["dy"] = torch.where(there[..., None], p["dy"], torch.zeros((), device="cuda"))
    pg = backward(p)
    for n in ("x", "dt", "B", "C", "z"):
        assert float((pg[n][there] - got[n][0]).abs().max()) <= 1e-5 * float(got[n].abs().max())
    assert float((pg["s0"] - got["s0"]).abs().max()) <= 1e-5 * float(got["s0"].abs().max())
    x = torch.where(there[..., None], c["x"][0][at], torch.zeros((), device="cuda"))
    pyc, _ = binding.causal_conv_fwd(x, c["w"], c["b"], initial_window=c["win"])
    assert torch.equal(pyc[there], yc[0])


def test_offsets_past_32_bits():
    """A row whose elements lie further apart than 2^31: strided views of a large buffer."""
    free, _ = torch.cuda.mem_get_info()
    step = (1 << 27) + 8  # elements between tokens; 20 tokens span 2.7e9 of them, 5.4 GB
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    buf = torch.empty(20 * step, dtype=torch.bfloat16, device="cuda")
    c, s = conv_inputs(1, 20, 16, 4, "bf16", 1), scan_inputs(1, 20, 16, 8, "bf16", 2)
    g = heads(1, 20, 2, 8, "bf16", 3, True)
    far = lambda t, at: torch.as_strided(buf, t.shape, (0, step, *t.stride()[2:]), at).copy_(t)  # noqa: E731
    fc = dict(c, x=far(c["x"], 0), dy=far(c["dy"], 16))
    assert all(torch.equal(a, b) for a, b in zip(conv_both(fc), conv_both(c)))
    names = ("x", "dt", "B", "C", "z", "dy")
    fs = dict(s, **{n: far(s[n], 32 + 16 * i) for i, n in enumerate(names)})
    assert all(torch.equal(a, b) for a, b in zip(scan_both(fs), scan_both(s)))
    fg = dict(g, x=far(g["x"], 160), g=far(g["g"], 176), dy=far(g["dy"], 192))
    assert torch.equal(binding.gated_norm_fwd(fg["x"], fg["g"], fg["w"]), binding.gated_norm_fwd(g["x"], g["g"], g["w"]))


def test_flags_by_their_truth():
    # steps that are positive without softplus, too: states grow past fp32 by negative ones
    c, s = conv_inputs(1, 9, 16, 4, "bf16", 1, states=False), scan_inputs(1, 9, 16, 8, "bf16", 2, soft=False)
    g = heads(1, 5, 2, 16, "bf16", 3, True)
    for yes, no in ((1, 0), ("x", ""), ([0], None)):
        f = lambda v: binding.causal_conv_fwd(c["x"], c["w"], silu=v)[0]  # noqa: E731
        assert torch.equal(f(yes), f(True)) and torch.equal(f(no), f(False)) and not torch.equal(f(yes), f(no))
        assert binding.causal_conv_fwd(c["x"], c["w"], output_final_window=no)[1] is None
        f = lambda v: forward(s, soft=v)[0]  # noqa: E731
        assert torch.equal(f(yes), f(True)) and torch.equal(f(no), f(False)) and not torch.equal(f(yes), f(no))
        for flag in ("gate_first", "sigmoid"):
            f = lambda v: binding.gated_norm_fwd(g["x"], g["g"], **{flag: v})  # noqa: E731, B023
            assert torch.equal(f(yes), f(True)) and torch.equal(f(no), f(False)) and not torch.equal(f(yes), f(no))


def test_pools_in_place_or_apart():
    """A pool that is read and another one that lies across it are refused; the same memory by another name is not."""
    c, s = conv_inputs(2, 1, 16, 4, "bf16", 1), scan_inputs(2, 1, 16, 8, "bf16", 2)
    wins, states = torch.zeros(5, 3, 16, device="cuda").bfloat16(), torch.zeros(5, 16, 8, device="cuda")
    step = lambda out, pool=wins: binding.causal_conv_step(c["x"][:, 0], c["w"], pool, c["b"], window_out=out)  # noqa: E731
    scan = lambda out, pool=states: binding.ssm_step(s["x"][:, 0], s["dt"][:, 0], s["A"], s["B"][:, 0], s["C"][:, 0], pool,  # noqa: E731
                                                     state_out=out)
    for call, pool in ((step, wins), (scan, states)):
        with pytest.raises(ValueError, match="share memory"):
            call(pool[1:], pool[:4])
        call(pool.view_as(pool))
        call(pool[3:], pool[:2])
