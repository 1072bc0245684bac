"""Host-side argument checks of the layer operators: nothing here reaches a
kernel, so these run without a GPU."""
import ctypes

import pytest
import torch

from gated_delta_rule_47_gb300 import binding, build

FAKE = 0x10000  # never dereferenced: every call below fails its checks first, or has nothing to do
BAD = ctypes.c_size_t(-1).value
F32, BF16 = binding.GDN_F32, binding.GDN_BF16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def fwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, o=FAKE, sf=None, cu=None, st=None, n=1, B=1, H=2, Hk=1, T=8, Dk=64,
             Dv=64, scale=1.0, flags=0, dtype=F32, ws=None, wsb=0)
    a.update(kw)
    return lib.linattn_chunk_fwd(*(a[x] for x in ("q", "k", "v", "g", "s0", "o", "sf", "cu", "st", "n", "B", "H", "Hk", "T",
                                                  "Dk", "Dv", "scale", "flags", "dtype", "ws", "wsb")), None)


def bwd(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, do=FAKE, dsf=None, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, ds0=None,
             cu=None, st=None, n=1, B=1, H=2, Hk=1, T=8, Dk=64, Dv=64, scale=1.0, flags=0, dtype=F32, ws=None, wsb=0)
    a.update(kw)
    return lib.linattn_chunk_bwd(*(a[x] for x in ("q", "k", "v", "g", "s0", "do", "dsf", "dq", "dk", "dv", "dg", "ds0", "cu",
                                                  "st", "n", "B", "H", "Hk", "T", "Dk", "Dv", "scale", "flags", "dtype",
                                                  "ws", "wsb")), None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_prompt_checks(lib, call):
    assert call(lib) == 4                            # no workspace
    assert call(lib, ws=FAKE + 8, wsb=1 << 30) == 4  # a misaligned one
    assert call(lib, q=None) == 1
    assert call(lib, dtype=9) == 1
    assert call(lib, flags=1) == 1                   # GDN_QK_L2NORM does not apply
    assert call(lib, B=-1) == 1
    assert call(lib, Hk=0) == 1
    assert call(lib, H=3, Hk=2) == 1
    assert call(lib, n=2) == 1                       # without offsets every row is a sequence
    assert call(lib, cu=FAKE, B=2, n=2) == 1         # packed rows
    assert call(lib, cu=FAKE, n=0) == 1              # tokens, but no sequence
    assert call(lib, Dk=96) == 2
    assert call(lib, H=70000, Hk=1) == 2
    assert call(lib, v=FAKE + 4) == 3
    odd = (ctypes.c_longlong * 15)(*[64 * 8] * 14, 1)
    odd[2] = 66
    assert call(lib, st=odd) == 3
    odd[2] = -64
    assert call(lib, st=odd) == 1
    assert call(lib, T=0, q=None, k=None) == 0       # nothing to do


def test_prompt_workspaces(lib):
    for f in (lib.linattn_chunk_fwd_workspace_bytes, lib.linattn_chunk_bwd_workspace_bytes):
        assert f(1, 4, 2, 100, 128, 128, 1, 0, 0, F32) not in (0, BAD)
        assert f(1, 4, 2, 0, 128, 128, 1, 0, 0, F32) == 0
        assert f(1, 4, 3, 100, 128, 128, 1, 0, 0, F32) == BAD
        assert f(1, 4, 2, 100, 32, 128, 1, 0, 0, F32) == BAD
        assert f(2, 4, 2, 100, 128, 128, 1, 0, 0, F32) == BAD  # two rows, one sequence
        assert f(1, 4, 2, 100, 128, 128, 7, 1, 0, F32) > f(1, 4, 2, 100, 128, 128, 1, 0, 0, F32)


def test_step_checks(lib):
    def plain(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, s=FAKE, so=FAKE, slots=FAKE, o=FAKE, B=1, H=2, Hk=1, Dk=64, Dv=64, n=4,
                 scale=1.0, flags=0, dtype=F32)
        a.update(kw)
        return lib.linattn_step(*a.values(), None)

    assert plain(q=None) == 1
    assert plain(flags=1) == 1
    assert plain(dtype=3) == 1
    assert plain(H=3, Hk=2) == 1
    assert plain(slots=None, B=5) == 1
    assert plain(Dv=256) == 2
    assert plain(s=FAKE + 8) == 3
    assert plain(B=0) == 0
    args = [FAKE] * 3 + [None] + [FAKE] * 5 + [1, 2, 1, 64, 64, 4, 1.0, 1, F32, None]
    assert lib.gdn_step(*args) == 1  # no beta


def test_norm_checks(lib):
    def f(x=FAKE, res=None, w=None, y=FAKE, s=FAKE, h=None, rows=2, C=256, group=0, eps=1e-6, e=1, dtype=BF16):
        return lib.rms_norm_fwd(x, res, w, y, s, h, rows, C, group, eps, e, dtype, None)

    assert f(x=None) == 1
    assert f(s=None) == 1
    assert f(eps=-1.0) == 1
    assert f(C=0) == 1
    assert f(group=100) == 1           # does not divide
    assert f(group=128, e=0) == 1      # groups are the 8-bit output's
    assert f(group=256) == 2
    assert f(C=1 << 20, group=128) == 2
    assert f(res=FAKE + 2) == 3
    assert f(rows=0) == 0
    assert lib.rms_norm_bwd(FAKE, FAKE, None, None, FAKE, None, 2, 256, 1e-6, BF16, None, 0, None) == 1
    assert lib.rms_norm_bwd_workspace_bytes(-1, 8) == BAD and lib.rms_norm_bwd_workspace_bytes(0, 8) == 0


def test_pool_checks(lib):
    assert lib.state_pool_copy(FAKE, 1, 4, 24, FAKE, FAKE, 1, None) == 3
    assert lib.state_pool_copy(FAKE + 8, 1, 4, 32, FAKE, FAKE, 1, None) == 3
    assert lib.state_pool_copy(None, 1, 4, 32, FAKE, FAKE, 1, None) == 1
    assert lib.state_pool_copy(FAKE, 1, 4, 32, None, FAKE, 1, None) == 1
    assert lib.state_pool_copy(FAKE, 1, 4, 32, None, None, 0, None) == 0
    assert lib.state_pool_fork(FAKE, 1, 4, 32, FAKE, FAKE, FAKE, 1, None, 0, None) == 4
    assert lib.state_pool_fork(FAKE, 1, 4, 32, None, FAKE, FAKE, 1, FAKE, 1 << 20, None) == 1
    assert lib.state_pool_free(None, 4, FAKE, 1, None) == 1
    assert lib.state_pool_compact(FAKE, 1, 4, 32, FAKE, FAKE, None, FAKE, 1 << 20, None) == 1
    assert lib.state_pool_compact(FAKE, 1, 4, 32, FAKE, FAKE, FAKE, None, 0, None) == 4
    assert lib.state_pool_fork_workspace_bytes(-1, 2) == BAD and lib.state_pool_compact_workspace_bytes(-1) == BAD


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        binding.rms_norm_fwd(x)
    with pytest.raises(TypeError):
        binding.state_pool_compact(torch.zeros(1, 2, 8), torch.zeros(2, dtype=torch.uint8))
    q = torch.zeros(1, 1, 4, 64)
    with pytest.raises(TypeError):
        binding.linattn_chunk_fwd(q, q, q, torch.zeros(1, 1, 4))
