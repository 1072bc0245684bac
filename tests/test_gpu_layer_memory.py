"""An allocation that fails raises torch's own error for it, whichever way a call takes."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [False, True])
def test_out_of_memory(stream):
    ensure_lib()
    s = torch.cuda.Stream() if stream else None
    x = torch.zeros(1 << 15, 1 << 13, device="cuda")  # 1 GB
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(x.device).total_memory
    try:  # torch's allocator gives no more than what is in use and a little
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (256 << 20)) / total)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            binding.rms_norm_fwd(x, stream=s)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            binding.rms_norm_bwd(x, x, stream=s)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    y, _, _ = binding.rms_norm_fwd(x, stream=s)
    torch.cuda.synchronize()
    assert not bool(y.any())
