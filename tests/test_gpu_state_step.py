"""Single-token steps against a pool of states: the CUDA kernels against the
recurrence in 64 bits.  Bounds on max|x - ref| / max|ref|: the library's
targets for o (1e-2 bf16, 1e-4 fp32); states are fp32 sums of exact products,
1e-5."""
import pytest
import torch

from gated_delta_rule_47_gb300 import binding
from gated_delta_rule_47_gb300.inputs import gdn_inputs
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, TOL_F32, ensure_lib, rel_err, to_dev

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def inputs(B, H, Hk, Dk, Dv, n_slots, dtype, seed, per_head=False):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    d = dict(q=unit(randn(B, Hk, Dk)), k=unit(randn(B, Hk, Dk)), v=randn(B, H, Dv), beta=torch.sigmoid(randn(B, H)))
    d = {n: x.to(DT[dtype]) for n, x in d.items()}
    d["g"] = torch.nn.functional.logsigmoid(randn(H) if per_head else randn(B, H)) / 4
    d["state"] = randn(n_slots, H, Dk, Dv)
    d = {n: x.cuda() for n, x in d.items()}
    d["slots"] = torch.randperm(n_slots, generator=gen)[:B].to(torch.int32).cuda()
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("delta,l2norm", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("B,H,Hk,Dk,Dv,per_head", [(1, 1, 1, 128, 128, False), (3, 4, 2, 64, 128, True),
                                                   (2, 6, 6, 128, 64, False), (5, 2, 1, 64, 64, False),
                                                   (40, 16, 8, 128, 128, False), (80, 8, 8, 64, 64, True)])
def test_step(B, H, Hk, Dk, Dv, per_head, delta, l2norm, dtype):
    d = inputs(B, H, Hk, Dk, Dv, B + 3, dtype, B + H, per_head)
    if l2norm:
        d["q"], d["k"] = 3 * d["q"], 2 * d["k"]
    slots = d["slots"].clone()
    if B > 2:
        slots[1], slots[2] = -1, B + 3  # idle rows
    want_o, want_s = ref.step(d["q"], d["k"], d["v"], d["g"], d["state"], slots, d["beta"] if delta else None, 0.6, l2norm)
    before, apart = d["state"].clone(), torch.full_like(d["state"], 7.0)
    args = (d["q"], d["k"], d["v"], *((d["beta"],) if delta else ()), d["g"])
    more = dict(l2norm=l2norm) if delta else {}
    f = binding.gdn_step if delta else binding.linattn_step
    o = f(*args, d["state"], slots=slots, state_out=apart, scale=0.6, **more)
    assert rel_err(o, want_o) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    assert torch.equal(d["state"], before)
    used = sorted(s for s in slots.tolist() if 0 <= s < B + 3)
    assert rel_err(apart[used], want_s[used]) <= 1e-5
    idle = [s for s in range(B + 3) if s not in used]
    assert bool((apart[idle] == 7.0).all())
    again = f(*args, d["state"], slots=slots, scale=0.6, **more)  # in place
    assert torch.equal(again, o) and torch.equal(d["state"][used], apart[used])
    assert torch.equal(d["state"][idle], before[idle])
    for b in range(B):
        if not 0 <= int(slots[b]) < B + 3:
            assert float(o[b].abs().max()) == 0.0


def test_without_slots_and_cleared():
    """No slots: page b; g = -inf starts a request over."""
    d = inputs(4, 2, 2, 128, 128, 6, "f32", 3)
    d["g"][2] = float("-inf")
    want_o, want_s = ref.step(d["q"], d["k"], d["v"], d["g"], d["state"])
    o = binding.linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"])
    assert rel_err(o, want_o) <= TOL_F32 and rel_err(d["state"], want_s) <= 1e-5


def test_steps_continue_a_prompt():
    """gdn_step from gdn_chunk_fwd's state gives gdn_chunk_fwd's next outputs,
    and linattn_step from linattn_chunk_fwd's."""
    B, H, T, D, n = 2, 4, 90, 128, 4
    d = to_dev(gdn_inputs(B, H, T + n, D, D, seed=5, dtype="bf16"))
    cut = {k: x[:, :, :T].contiguous() for k, x in d.items()}
    whole, _ = binding.gdn_chunk_fwd(d["q"], d["k"], d["v"], d["beta"], d["g"])
    _, state = binding.gdn_chunk_fwd(cut["q"], cut["k"], cut["v"], cut["beta"], cut["g"], output_final_state=True)
    lin, _ = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"])
    _, lin_state = binding.linattn_chunk_fwd(cut["q"], cut["k"], cut["v"], cut["g"], output_final_state=True)
    for t in range(T, T + n):
        q, k, v, beta, g = (d[x][:, :, t].contiguous() for x in ("q", "k", "v", "beta", "g"))
        o = binding.gdn_step(q, k, v, beta, g, state)
        assert rel_err(o, whole[:, :, t].double().cpu().numpy()) <= 2 * TOL_BF16  # both sides carry the bound
        o = binding.linattn_step(q, k, v, g, lin_state)
        assert rel_err(o, lin[:, :, t].double().cpu().numpy()) <= 2 * TOL_BF16


def test_refusals():
    d = inputs(2, 4, 2, 64, 64, 3, "bf16", 1)
    f = binding.linattn_step
    with pytest.raises(TypeError):
        f(d["q"], d["k"], d["v"], d["g"], d["state"].bfloat16())
    with pytest.raises(TypeError):
        f(d["q"].half(), d["k"].half(), d["v"].half(), d["g"], d["state"])
    with pytest.raises(TypeError):
        f(d["q"], d["k"], d["v"], d["g"], d["state"], slots=d["slots"].long())
    with pytest.raises(ValueError):
        f(d["q"], d["k"], d["v"], d["g"], d["state"], slots=d["slots"][:1])
    with pytest.raises(ValueError):
        f(d["q"], d["k"], d["v"], d["g"], d["state"][:1])
    with pytest.raises(ValueError):
        f(d["q"], d["k"], d["v"][:, :3].contiguous(), d["g"][:, :3].contiguous(), d["state"][:, :3].contiguous())
    with pytest.raises(ValueError):
        binding.gdn_step(d["q"], d["k"], d["v"], d["beta"][:1], d["g"], d["state"])
    with pytest.raises(binding.GdnError):  # Dk = 32
        s = torch.zeros(3, 4, 32, 64, device="cuda")
        f(d["q"][..., :32].contiguous(), d["k"][..., :32].contiguous(), d["v"], d["g"], s)
