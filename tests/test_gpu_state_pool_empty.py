"""Pools that hold no bytes (no layers, no slots, pages of nothing): the marks,
children and new places are those of any other pool, and there is nothing to move."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def idx(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("shape", [(0, 8, 4), (1, 8, 0), (2, 8, 0, 4)])
def test_no_bytes(shape):
    pool = torch.zeros(*shape, device="cuda")
    live = torch.tensor([1, 0, 0, 1, 0, 0, 1, 1], dtype=torch.uint8, device="cuda")
    binding.state_pool_copy(pool, idx(0), idx(1))
    assert binding.state_pool_fork(pool, live, idx(3, -1, 2)).tolist() == [1, 2, -1]
    assert live.tolist() == [1, 1, 1, 1, 0, 0, 1, 1]
    remap, n = binding.state_pool_compact(pool, live)
    assert remap.tolist() == [0, 1, 2, 3, -1, -1, 4, 5] and int(n) == 6
    assert live.tolist() == [1] * 6 + [0] * 2


@pytest.mark.parametrize("layers", [0, 1, 3])
def test_no_slots(layers):
    pool, live = torch.zeros(layers, 0, 4, device="cuda"), torch.zeros(0, dtype=torch.uint8, device="cuda")
    binding.state_pool_copy(pool, idx(0), idx(0))
    assert binding.state_pool_fork(pool, live, idx(-1, 0)).tolist() == [-1, -1]
    remap, n = binding.state_pool_compact(pool, live)
    assert remap.numel() == 0 and int(n) == 0
