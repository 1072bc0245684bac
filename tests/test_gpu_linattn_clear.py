"""Decays that clear the state, with states going in and coming out: the bounds
on fp32 outputs (dg 1e-4, states and their gradients 1e-5; see
test_gpu_linattn.py) hold where the state before is dropped, too."""
import pytest

from gated_delta_rule_47_gb300 import binding
from tests import layer_reference as ref
from tests.gpu_util import TOL_BF16, TOL_F32, ensure_lib, rel_err
from tests.test_gpu_linattn import inputs, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,simt", [("bf16", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("H,Hk,lens", [(2, 2, None), (4, 2, None), (2, 1, [90, 1, 209])])
def test_cleared(H, Hk, lens, states, dtype, simt):
    ensure_lib()
    d = inputs(1, H, Hk, 300, 128, 128, dtype, 17, lens)
    d["g"][:, :, 130] = float("-inf")
    d["g"][:, 1, 200:280] = -40.0
    d["g"][:, 0, :3] = float("-inf")
    s0, dsf = (d["s0"], d["dsf"]) if states else (None, None)
    cu = None if lens is None else offsets(lens)
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    o, sf = binding.linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=s0, output_final_state=True,
                                      cu_seqlens=cu, simt=simt)
    ro, rs = ref.linattn(d["q"], d["k"], d["v"], d["g"], s0, lens)
    assert rel_err(o, ro) <= tol and rel_err(sf, rs) <= 1e-5
    got = binding.linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], initial_state=s0, dfinal_state=dsf,
                                    cu_seqlens=cu, simt=simt)
    want = ref.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], s0, dsf, lens)
    for name, x, r, t in zip(("dq", "dk", "dv", "dg", "ds0"), got, want, (tol, tol, tol, 1e-4, 1e-5)):
        assert (x is None and not states) or rel_err(x, r) <= t, name
