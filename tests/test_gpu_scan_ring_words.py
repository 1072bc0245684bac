"""What a workspace held before the tensor-core scans' ring lies in it: pairs of 32-bit
numbers of which each in turn was once a launch's tag count as none."""
import torch

import pytest

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("first", [-4194304, 0])
def test_negative_whole_numbers_and_nan_in_the_workspace(first):
    """Words whose upper halves are the 32,768 numbers from `first` on (as fp32, NaN from -4194304), 512 of them a
    launch: one of these launches has the number that a 32-bit tag from there on would give it."""
    gen = torch.Generator().manual_seed(5)
    shape = (1, 64, 640, 128)
    q, k = (torch.nn.functional.normalize(torch.randn(shape, generator=gen), dim=-1).bfloat16().cuda() for _ in range(2))
    v = torch.randn(shape, generator=gen).bfloat16().cuda()
    beta, g = torch.rand(shape[:3], generator=gen).bfloat16().cuda(), -torch.rand(shape[:3], generator=gen).cuda() / 16
    ws = torch.zeros(binding.workspace_bytes(1, 64, 640, 128, 128), dtype=torch.uint8, device="cuda")
    want = binding.gdn_chunk_fwd(q, k, v, beta, g, workspace=ws)[0].clone()
    words = ws[: ws.numel() // 16 * 16].view(torch.int32).view(-1, 4)  # a slot's tag takes 16 bytes
    number = torch.arange(len(words), device="cuda", dtype=torch.int32) % 512
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(64):
        words[:, 0] = words[:, 2] = 3000
        words[:, 1] = words[:, 3] = first + 512 * i + number
        differ += (binding.gdn_chunk_fwd(q, k, v, beta, g, workspace=ws)[0] != want).any()
    assert int(differ) == 0 and binding.device_error() == 0
