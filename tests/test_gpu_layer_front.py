"""The layer operators' two ways in: the short one and, for a call on a given
stream, the long one launch the same kernels on the same arguments, so their
outputs are equal bit for bit; and what the short one declines or the library
refuses still raises."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_linattn import inputs, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def both(call):
    short = call(None)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    long = call(stream)
    torch.cuda.synchronize()
    for x, y in zip(*((r if isinstance(r, tuple) else (r,)) for r in (short, long))):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype == y.dtype and x.stride() == y.stride()
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,per_head,token_major", [(None, False, False), (None, True, True), ([100, 0, 160], False, True)])
def test_prompts(dtype, lens, per_head, token_major):
    d = inputs(1 if lens else 2, 4, 2, 260, 128, 64, dtype, 3, lens, per_head, token_major=token_major)
    cu = None if lens is None else offsets(lens)
    both(lambda s: binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], scale=0.5,
                                             output_final_state=True, cu_seqlens=cu, stream=s))
    both(lambda s: binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, stream=s))
    both(lambda s: binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=d["s0"],
                                             dfinal_state=d["dsf"], cu_seqlens=cu, scale=0.5, stream=s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps(dtype):
    q, k, v = (torch.randn(3, n, 64, device="cuda").to(dtype) for n in (2, 2, 4))
    g, beta = -torch.rand(3, 4, device="cuda"), torch.rand(3, 4, device="cuda").to(dtype)
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    pool = torch.randn(5, 4, 64, 64, device="cuda")
    for more in ({}, dict(slots=slots)):
        both(lambda s: binding.linattn_step(q, k, v, g, pool, state_out=torch.empty_like(pool), scale=0.3, stream=s, **more))
        both(lambda s: binding.gdn_step(q, k, v, beta, g[0], pool, state_out=torch.empty_like(pool), l2norm=True, stream=s, **more))

    def in_place(s):
        state = pool.clone()
        torch.cuda.synchronize()
        return binding.gdn_step(q, k, v, beta, g, state, slots=slots, stream=s), state
    both(in_place)


@pytest.mark.parametrize("out,group", [(None, 0), (torch.float8_e4m3fn, 0), (torch.float8_e4m3fn, 64)])
def test_norms(out, group):
    x, res = torch.randn(2, 5, 192, device="cuda").bfloat16(), torch.randn(2, 5, 192, device="cuda").bfloat16()
    w = torch.rand(192, device="cuda")
    both(lambda s: binding.rms_norm_fwd(x, w, residual=res, eps=1e-5, out_dtype=out, group=group, stream=s))
    both(lambda s: binding.rms_norm_fwd(x, out_dtype=out, group=group, stream=s)[:2])
    both(lambda s: binding.rms_norm_bwd(x, res, w, dresidual=x, stream=s))
    both(lambda s: binding.rms_norm_bwd(x, res, stream=s))


def test_pools():
    start = torch.randn(2, 6, 4, 8, device="cuda")
    parents = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")

    def call(s):
        pool, live = start.clone(), torch.tensor([0, 1, 0, 0, 1, 0], dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        children = binding.state_pool_fork(pool, live, parents, stream=s)
        remap, n = binding.state_pool_compact(pool, live, stream=s)
        return children, remap, n, live, pool[:, :3]
    both(call)


def test_what_is_declined_or_refused():
    x = torch.randn(4, 256, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        binding.rms_norm_fwd(x.half())
    with pytest.raises(TypeError):
        binding.rms_norm_fwd(x, out_dtype=torch.float16)
    with pytest.raises((TypeError, ValueError)):
        binding.rms_norm_fwd(x, torch.rand(8, device="cuda"))
    with pytest.raises(binding.GdnError):
        binding.rms_norm_fwd(x, eps=-1.0)
    with pytest.raises(binding.GdnError):  # sizes the library does not have
        binding.linattn_step(*(torch.randn(1, 1, 32, device="cuda") for _ in range(3)), torch.zeros(1, 1, device="cuda"),
                             torch.zeros(1, 1, 32, 32, device="cuda"))
