"""Pages of the pool of recurrent states: every result is exact."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def make(layers, slots, page, live, seed, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    pool = torch.randn(layers, slots, *page, generator=gen).to(dtype).cuda()
    mask = torch.zeros(slots, dtype=torch.uint8)
    mask[torch.randperm(slots, generator=gen)[:live]] = 1
    return pool, mask.cuda(), gen


def idx(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layers,slots,page,dtype", [(1, 8, (4,), torch.float32), (3, 9, (2, 64, 64), torch.float32),
                                                     (2, 20, (16, 128, 128), torch.float32), (2, 7, (5, 8), torch.bfloat16)])
def test_copy(layers, slots, page, dtype):
    pool, _, _ = make(layers, slots, page, 3, 1, dtype)
    want = pool.clone()
    binding.state_pool_copy(pool, idx(0, 2, -1, 5, 6, -2, slots), idx(1, 3, 4, -1, slots, 5, 5))
    want[:, 1], want[:, 3], want[:, 4] = want[:, 0], want[:, 2], 0
    assert torch.equal(pool, want)
    binding.state_pool_copy(pool, idx(), idx())
    assert torch.equal(pool, want)


@pytest.mark.parametrize("layers,slots,page,live,n", [(1, 4, (4,), 1, 2), (2, 64, (2, 64, 64), 40, 30), (1, 3000, (8,), 1200, 2100),
                                                      (3, 6, (16, 128, 64), 6, 3), (1, 5, (4,), 0, 3)])
def test_fork(layers, slots, page, live, n):
    pool, mask, gen = make(layers, slots, page, live, 2)
    parents = torch.randint(-2, slots + 1, (n,), generator=gen).to(torch.int32)
    want, want_live, free = pool.clone(), mask.cpu().tolist(), [s for s in range(slots) if not mask[s]]
    alive, children = list(want_live), []
    for p in parents.tolist():
        if (p == -1 or (0 <= p < slots and alive[p])) and free:
            c = free.pop(0)
            want[:, c] = pool[:, p] if p >= 0 else 0
            want_live[c] = 1
            children.append(c)
        else:
            children.append(-1)
    got = binding.state_pool_fork(pool, mask, parents.cuda())
    assert got.tolist() == children
    assert mask.tolist() == want_live and torch.equal(pool, want)


@pytest.mark.parametrize("layers,slots,page,live", [(1, 1, (4,), 1), (1, 1, (4,), 0), (2, 9, (2, 64, 64), 4), (1, 40, (16,), 40),
                                                    (1, 40, (16,), 0), (1, 2500, (8,), 1201), (3, 31, (4, 128, 128), 17)])
def test_compact(layers, slots, page, live):
    pool, mask, _ = make(layers, slots, page, live, 3)
    before, alive = pool.clone(), [s for s in range(slots) if mask[s]]
    remap, n = binding.state_pool_compact(pool, mask)
    holes = [s for s in range(live) if s not in alive]
    want = {s: s for s in alive if s < live}
    want.update(zip([s for s in alive if s >= live], holes))
    assert int(n) == live
    assert remap.tolist() == [want.get(s, -1) for s in range(slots)]
    assert mask.tolist() == [1] * live + [0] * (slots - live)
    for s, t in want.items():
        assert torch.equal(pool[:, t], before[:, s])


def test_free_and_reuse():
    pool, mask, _ = make(2, 10, (2, 64), 10, 4)
    binding.state_pool_free(mask, idx(3, 7, 3, -1, 10, 99))
    assert mask.tolist() == [1, 1, 1, 0, 1, 1, 1, 0, 1, 1]
    children = binding.state_pool_fork(pool, mask, idx(0, -1, 5))
    assert children.tolist() == [3, 7, -1] and int(mask.sum()) == 10
    assert torch.equal(pool[:, 3], pool[:, 0]) and float(pool[:, 7].abs().max()) == 0.0


def test_offsets_past_32_bits():
    """A pool of 4.3 GB of 16-bit words: page addresses pass 2^32 bytes."""
    pool = torch.zeros(2, 70, 64 * 1024, 256, dtype=torch.bfloat16, device="cuda")
    pool[1, 68] = 3.0
    binding.state_pool_copy(pool, idx(68), idx(69))
    assert bool((pool[1, 69] == 3.0).all()) and float(pool[0].abs().max()) == 0.0


def test_refusals():
    pool, mask, _ = make(1, 8, (4,), 3, 1)
    with pytest.raises(TypeError):
        binding.state_pool_copy(pool.cpu(), idx(0), idx(1))
    with pytest.raises(ValueError):
        binding.state_pool_copy(pool[:, ::2], idx(0), idx(1))
    with pytest.raises(ValueError):
        binding.state_pool_copy(pool, idx(0, 1), idx(1))
    with pytest.raises(TypeError):
        binding.state_pool_copy(pool, idx(0).long(), idx(1))
    with pytest.raises(ValueError):  # 12-byte pages
        binding.state_pool_copy(pool[..., :3].contiguous(), idx(0), idx(1))
    with pytest.raises(ValueError):
        binding.state_pool_fork(pool, mask[:4], idx(0))
    with pytest.raises(TypeError):
        binding.state_pool_compact(pool, mask.int())
