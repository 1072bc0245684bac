"""The layer operators inside a captured graph: replays on new inputs give what
the calls give."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_linattn import inputs, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_decoding_step():
    """Norm and step, the state updated in place, three replays against three calls."""
    x, res = (torch.randn(4, 512, device="cuda").bfloat16() for _ in range(2))
    q, k = (torch.randn(4, 2, 128, device="cuda").bfloat16() / 11 for _ in range(2))
    v, beta = torch.randn(4, 4, 128, device="cuda").bfloat16(), torch.rand(4, 4, device="cuda").bfloat16()
    g, pool = -torch.rand(4, 4, device="cuda"), torch.randn(6, 4, 128, 128, device="cuda")
    slots = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device="cuda")

    def step(state):
        y, s, h = binding.rms_norm_fwd(x, residual=res, out_dtype=torch.float8_e4m3fn, group=128)
        return y.view(torch.uint8), s, h, binding.gdn_step(q, k, v, beta, g, state, slots=slots, l2norm=True)

    captured, called = pool.clone(), pool.clone()
    step(pool.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(captured)
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        q.copy_(torch.randn_like(q))
        graph.replay()
        want = step(called)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        assert torch.equal(captured, called)


@pytest.mark.parametrize("T,lens", [(300, [100, 200]), (6000, [5000, 1000]), (4000, None)])
def test_prompts_and_gradients(T, lens):
    """Also calls whose sequences are cut into pieces (counters and flags are set anew by each replay)."""
    d = inputs(1, 2, 1, T, 128, 128, "bf16", 3, lens)
    cu = None if lens is None else offsets(lens)

    def call():
        o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], output_final_state=True,
                                          cu_seqlens=cu)
        return o, sf, *binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["s0"],
                                                 dfinal_state=d["dsf"], cu_seqlens=cu)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        d["v"].copy_(torch.randn_like(d["v"]))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    assert binding.device_error() == 0
