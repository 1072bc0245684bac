"""A row of more than 2^28 tokens (34 GB a tensor): its sequences lie past 2^34
elements, and there are more 16-byte words of tokens of no sequence than 2^31."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


def test_forward():
    ensure_lib()
    T, cut = (1 << 28) + 4000, 400
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    x, o = torch.empty(1, 1, T, 64, dtype=torch.bfloat16, device="cuda"), torch.full((1, 1, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x[:, :, -cut:] = (torch.randn(1, 1, cut, 64, generator=torch.Generator().manual_seed(1)) / 8).bfloat16().cuda()
    g = torch.full((1,), -0.02, device="cuda")
    cu = torch.tensor([T - 300, T - 170, T - 100], dtype=torch.int32, device="cuda")
    _, sf = binding.linattn_chunk_fwd(x, x, x, g, output_final_state=True, cu_seqlens=cu, o=o)
    near = x[:, :, -cut:].contiguous()
    want, want_sf = binding.linattn_chunk_fwd(near, near, near, g, output_final_state=True, cu_seqlens=cu - (T - cut))
    assert torch.equal(o[:, :, -cut:], want) and torch.equal(sf, want_sf)
    assert not any(bool(part.any()) for part in o[:, :, :-300].reshape(-1).view(torch.int64).split(1 << 30))
    assert binding.device_error() == 0
    del x, o
    torch.cuda.empty_cache()
