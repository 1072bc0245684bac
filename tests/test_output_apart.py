"""Which outputs of the caller's a call refuses because they lie over what it reads:
memory in common, not the span between a first and a last element."""
import random

import pytest
import torch

from gated_delta_rule_47_gb300 import binding


def shares(a, b):
    try:
        binding._apart(a, b, "a and b")
        return False
    except ValueError:
        return True


def bytes_of(t):
    size, out = t.element_size(), set()
    for index in torch.cartesian_prod(*(torch.arange(n) for n in t.shape)).reshape(-1, t.dim()).tolist():
        at = t.data_ptr() + size * sum(i * s for i, s in zip(index, t.stride()))
        out.update(range(at, at + size))
    return out


def test_columns_of_one_buffer():
    buf = torch.zeros(2, 5, 48, dtype=torch.bfloat16)
    assert not shares(buf[..., :16], buf[..., 16:48]) and not shares(buf[..., 16:48], buf[..., :16])
    assert not shares(buf[..., :8], buf[:, 1:3, 40:]) and not shares(buf[0, :, :8], buf[1, :, 8:])
    assert shares(buf[..., :16], buf[..., 8:24]) and shares(buf[..., 32:], buf[..., 40:48])
    assert shares(buf, buf) and shares(buf[..., :16], buf)
    assert not shares(buf[0], buf[1]) and shares(buf[0, 0], buf[0])
    pool = torch.zeros(6, 3, 16)
    assert shares(pool[1:], pool[:5]) and not shares(pool[:3], pool[3:]) and shares(pool[:2], pool[1:3])


@pytest.mark.parametrize("seed", range(300))
def test_never_lets_common_memory_pass(seed):
    """Any two views of a buffer, one of them in elements of twice the size: if bytes are common, it is seen."""
    rng = random.Random(seed)
    buf = torch.zeros(400, dtype=torch.bfloat16)
    views = []
    for t in (buf, buf.view(torch.float32) if rng.random() < 0.3 else buf):
        width = rng.choice([1, 2, 4, 6])
        step = rng.choice([0, width, 8, 12, 16])
        shape, stride = (rng.randint(1, 3), rng.randint(1, 4), width), (rng.choice([0, step * 2, 24, 32]), step, 1)
        most = sum((n - 1) * s for n, s in zip(shape, stride)) + 1
        views.append(torch.as_strided(t, shape, stride, rng.randint(0, min(t.numel() - most, 40))))
    a, b = views
    if bytes_of(a) & bytes_of(b):
        assert shares(a, b) and shares(b, a)
