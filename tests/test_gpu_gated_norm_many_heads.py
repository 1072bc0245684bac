"""The gated norm's backward with a weight for each of so many heads that the last
columns' numbers, rounded up to 32, pass 32 bits: the columns are summed all the
same.  One token, so a head's dweight is its dy n(x) act(gate)."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib
from tests.test_gpu_gated_norm import close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()
    yield
    torch.cuda.empty_cache()  # later tests ask how much is free


def test_columns_up_to_the_last():
    H, D = (1 << 28) - 1, 8
    free, _ = torch.cuda.mem_get_info()
    if free < 64 << 30:
        pytest.skip("needs 64 GB")
    x = torch.empty(1, 1, H, D, dtype=torch.bfloat16, device="cuda")
    w = torch.full((H, D), 2.0, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    some = torch.cat([torch.arange(40), torch.randint(0, H, (1000,)), torch.arange(H - 40, H)]).cuda()
    x.fill_(1.0)
    gate, dy = x, x.clone()  # the gate's values are x's
    x[0, 0, some], dy[0, 0, some] = (torch.randn(len(some), D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    dx, dg, dw = binding.gated_norm_bwd(dy, x, gate, w)
    assert dw.shape == (H, D)
    u, t = x[0, 0, some].double(), dy[0, 0, some].double()
    want = t * u / ((u * u).mean(-1, keepdim=True) + 1e-6).sqrt() * u / (1 + torch.exp(-u))
    close(dw[some], want.cpu(), "f32")
    # every other head's is that of ones
    one = torch.tensor(1.0, dtype=torch.float64)
    each = float(one / (1 + 1e-6) ** 0.5 / (1 + torch.exp(-one)))
    dw[some] = each
    assert float(dw.sub_(each).abs_().max()) <= 1e-5
    assert bool(dx[0, 0, -1].isfinite().all()) and bool(dg[0, 0, -1].isfinite().all())
