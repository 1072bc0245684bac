"""Gradients of views whose elements share memory (sliding windows over one
row): as those of their copies, bit for bit."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,simt", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)])
@pytest.mark.parametrize("stream", [False, True])
def test_windows(dtype, simt, stream):
    ensure_lib()
    B, H, T, D = 1, 2, 150, 64
    gen = torch.Generator().manual_seed(3)
    row = 64 * H + 16 * T + D  # token t of head h starts at 64 h + 16 t
    base = (torch.randn(4 * row, generator=gen) / 8).cuda().to(dtype)
    q, k, v, do = (base.as_strided((B, H, T, D), (row, 64, 16, 1), i * row) for i in range(4))
    g = (-torch.rand(T + H, generator=gen)).cuda().as_strided((B, H, T), (T + H, 1, 1))
    s = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    got = binding.linattn_chunk_bwd(q, k, v, g, do, simt=simt, stream=s)
    want = binding.linattn_chunk_bwd(*(x.contiguous() for x in (q, k, v, g, do)), simt=simt)
    torch.cuda.synchronize()
    for x, y in zip(got[:4], want):
        assert torch.equal(x, y)
