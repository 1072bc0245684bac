"""The ring of the tensor-core scans: a slot's bytes are seen before its tag.  Launches
on the same inputs give equal bits (nothing in them depends on an order), back to
back and with the device idle between them; a slot that was read before its bytes
had arrived gave some head other tokens in up to half of them."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from gated_delta_rule_47_gb300.inputs import WORKLOADS
from tests.gpu_util import ensure_lib, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("idle", [False, True])
@pytest.mark.parametrize("name", ["gdn_b4h16t4096d128_bf16", "deltaproduct_r2_b4h16t4096d128_bf16"])
def test_equal_launches_give_equal_bits(name, idle):
    w = WORKLOADS[name]
    d = to_dev(w.make())
    f = binding.deltaproduct_chunk_fwd if name.startswith("delta") else binding.gdn_chunk_fwd
    first = f(d["q"], d["k"], d["v"], d["beta"], d["g"], chunk=w.chunk)[0].clone()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        if idle:
            torch.cuda.synchronize()
        differ += (f(d["q"], d["k"], d["v"], d["beta"], d["g"], chunk=w.chunk)[0] != first).any()
    assert int(differ) == 0 and binding.device_error() == 0


def test_whole_numbers_in_the_workspace_are_no_tags():
    """A workspace that held pairs of small whole numbers (offsets, lengths beside sequence numbers): none of
    them counts as a tag, whichever number of launches the process has made."""
    gen = torch.Generator().manual_seed(3)
    q, k = (torch.nn.functional.normalize(torch.randn(1, 2, 640, 128, generator=gen), dim=-1).bfloat16().cuda() for _ in range(2))
    v = torch.randn(1, 2, 640, 128, generator=gen).bfloat16().cuda()
    beta, g = torch.rand(1, 2, 640, generator=gen).bfloat16().cuda(), -torch.rand(1, 2, 640, generator=gen).cuda() / 16
    ws = torch.zeros(binding.workspace_bytes(1, 2, 640, 128, 128), dtype=torch.uint8, device="cuda")
    first = binding.gdn_chunk_fwd(q, k, v, beta, g, workspace=ws)[0].clone()
    room = ws[: ws.numel() // 8 * 8].view(torch.int32).view(-1, 2)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(3000):
        room[:, 0], room[:, 1] = 1000, 3000  # the launch of that number would take every slot for filled
        differ += (binding.gdn_chunk_fwd(q, k, v, beta, g, workspace=ws)[0] != first).any()
    assert int(differ) == 0 and binding.device_error() == 0
