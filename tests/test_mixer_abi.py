"""Host-side argument checks of the operators next to a mixer: nothing here reaches a
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


def strides(*x):
    return (ctypes.c_longlong * len(x))(*x)


def call(f, given, kw, stream=None):
    assert set(kw) <= set(given), kw
    return f(*{**given, **kw}.values(), stream)


def test_conv_checks(lib):
    def fwd(**kw):
        a = dict(x=FAKE, w=FAKE, b=None, win=None, y=FAKE, out=None, cu=None, st=None, n=1, B=1, T=8, C=16, W=4, flags=32, dtype=BF16)
        return call(lib.causal_conv_fwd, a, kw)

    def bwd(**kw):
        a = dict(x=FAKE, w=FAKE, b=None, dy=FAKE, win=None, dout=None, dx=FAKE, dw=FAKE, db=None, dwin=None, cu=None, st=None, n=1,
                 B=1, T=8, C=16, W=4, flags=32, dtype=BF16, ws=None, wsb=0)
        return call(lib.causal_conv_bwd, a, kw)

    for f in (fwd, bwd):
        assert f(x=None) == 1
        assert f(w=None) == 1
        assert f(dtype=9) == 1
        assert f(flags=1) == 1
        assert f(B=-1) == 1
        assert f(n=2) == 1                    # without offsets every row is a sequence
        assert f(cu=FAKE, B=2, n=2) == 1      # packed rows
        assert f(cu=FAKE, n=0) == 1           # tokens, but no sequence
        assert f(W=5) == 2 and f(W=1) == 2
        assert f(C=12) == 2
        assert f(B=70000, n=70000) == 2
        assert f(B=60000, n=60000, T=60000) == 2
        assert f(x=FAKE + 8) == 3 and f(win=FAKE + 2) == 3
        assert f(st=strides(128, 20, 128, 16)) == 3
        assert f(st=strides(128, -16, 128, 16)) == 1
    assert fwd(st=strides(128, 16, 128, 8)) == 1  # rows of y in one place
    assert fwd(T=0, x=None, y=None) == 0
    assert bwd() == 4 and bwd(ws=FAKE + 8, wsb=1 << 30) == 4 and bwd(ws=FAKE, wsb=8) == 4
    assert bwd(dw=None) == 1
    q = lib.causal_conv_bwd_workspace_bytes
    assert q(1, 100, 64, 4) not in (0, BAD) and q(1, 0, 64, 4) == 0
    assert q(-1, 8, 8, 4) == BAD and q(1, 8, 8, 9) == BAD and q(1, 8, 6, 4) == BAD

    def step(**kw):
        a = dict(x=FAKE, w=FAKE, b=None, win=FAKE, out=FAKE, slots=FAKE, y=FAKE, sx=16, B=2, C=16, W=4, n=4, flags=0, dtype=BF16)
        return call(lib.causal_conv_step, a, kw)

    assert step(win=None) == 1 and step(flags=64) == 1 and step(slots=None, B=5) == 1 and step(n=-1) == 1
    assert step(W=7) == 2 and step(C=20) == 2 and step(sx=12) == 3 and step(sx=-16) == 1 and step(y=FAKE + 4) == 3
    assert step(B=0) == 0


def test_scan_checks(lib):
    def fwd(**kw):
        a = dict(x=FAKE, dt=FAKE, A=FAKE, B_=FAKE, C_=FAKE, D=None, z=None, b=None, s0=None, y=FAKE, sf=None, cu=None, st=None, n=1,
                 B=1, T=4000, Di=16, N=16, flags=16, dtype=F32, ws=None, wsb=0)
        return call(lib.ssm_scan_fwd, a, kw)

    def bwd(**kw):
        a = dict(x=FAKE, dt=FAKE, A=FAKE, B_=FAKE, C_=FAKE, D=None, z=None, b=None, s0=None, dy=FAKE, dsf=None, dx=FAKE, ddt=FAKE,
                 dA=FAKE, dB=FAKE, dC=FAKE, dD=None, dz=None, db=None, ds0=None, cu=None, st=None, n=1, B=1, T=4000, Di=16, N=16,
                 flags=16, dtype=F32, ws=None, wsb=0)
        return call(lib.ssm_scan_bwd, a, kw)

    for f in (fwd, bwd):
        assert f() == 4 and f(ws=FAKE + 8, wsb=1 << 40) == 4 and f(ws=FAKE, wsb=16) == 4
        for name in ("x", "dt", "A", "B_", "C_"):
            assert f(**{name: None}) == 1 and f(**{name: FAKE + 4}) == 3
        assert f(dtype=2) == 1 and f(flags=8) == 1 and f(T=-1) == 1 and f(n=3) == 1 and f(cu=FAKE, n=0) == 1
        assert f(N=64) == 2 and f(N=12) == 2 and f(Di=18) == 2 and f(dtype=BF16, Di=12) == 2
        assert f(st=strides(*[16] * 11, 6)) in (1, 3) and f(st=strides(*[-16] * 12)) == 1
    assert fwd(st=strides(*[16] * 11, 8)) == 1
    assert bwd(z=FAKE) == 1               # the gate's gradient has no place
    assert bwd(dA=None) == 1
    assert fwd(T=0, x=None) == 0
    for q in (lib.ssm_scan_fwd_workspace_bytes, lib.ssm_scan_bwd_workspace_bytes):
        assert q(1, 4000, 64, 16, F32) not in (0, BAD) and q(1, 0, 64, 16, F32) == 0
        assert q(1, 40, 64, 24, F32) == BAD and q(-1, 40, 64, 16, F32) == BAD and q(1, 40, 12, 16, BF16) == BAD

    def step(**kw):
        a = dict(x=FAKE, dt=FAKE, A=FAKE, B_=FAKE, C_=FAKE, D=None, z=None, b=None, s=FAKE, so=FAKE, slots=FAKE, y=FAKE, st=None,
                 B=2, Di=16, N=16, n=4, flags=0, dtype=F32)
        return call(lib.ssm_step, a, kw)

    assert step(s=None) == 1 and step(flags=32) == 1 and step(slots=None, B=5) == 1
    assert step(N=4) == 2 and step(Di=10) == 2 and step(so=FAKE + 4) == 3
    assert step(st=strides(16, 16, 6, 16, 16)) == 3 and step(st=strides(16, 16, 16, -16, 16)) == 1
    assert step(B=0) == 0


def test_norm_checks(lib):
    def gated(**kw):
        a = dict(x=FAKE, g=FAKE, w=None, y=FAKE, st=None, B=1, T=4, H=2, D=64, eps=1e-6, flags=256, dtype=BF16)
        return call(lib.gated_norm_fwd, a, kw)

    def gated_back(**kw):
        a = dict(dy=FAKE, x=FAKE, g=FAKE, w=None, dx=FAKE, dg=FAKE, dw=FAKE, st=None, B=1, T=4, H=2, D=64, eps=1e-6, flags=256,
                 dtype=BF16, ws=None, wsb=0)
        return call(lib.gated_norm_bwd, a, kw)

    for f, n in ((gated, 6), (gated_back, 12)):
        assert f(x=None) == 1 and f(g=None) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and f(flags=2) == 1
        assert f(D=20) == 2 and f(D=16384) == 2 and f(B=1 << 20, T=1 << 20) == 2 and f(T=1, H=1 << 20, D=8192) == 2 and f(g=FAKE + 8) == 3
        assert f(st=strides(*[4] * n)) == 3 and f(st=strides(*[-64] * n)) == 1
    assert gated(T=0) == 0
    assert gated_back() == 4 and gated_back(dw=None) == 1
    assert gated_back(ws=FAKE, wsb=1 << 30, st=strides(*[512, 128, 64] * 3, 512, 32, 64)) == 1  # dx's elements in one place
    assert lib.gated_norm_bwd_workspace_bytes(1, 4, 2, 64, 0) not in (0, BAD)
    assert lib.gated_norm_bwd_workspace_bytes(1, 4, 2, 66, 0) == BAD

    def block(**kw):
        a = dict(x=FAKE, res=FAKE, w1=None, s=None, w2=None, y=FAKE, h=FAKE, rows=6, C=64, groups=0, eps=1e-6, dtype=BF16)
        return call(lib.block_norm_fwd, a, kw)

    def block_back(**kw):
        a = dict(dy=FAKE, dh=None, x=FAKE, h=FAKE, w1=None, s=None, w2=None, dx=FAKE, dr=FAKE, dw1=None, ds=None, dw2=None, rows=6,
                 C=64, groups=0, eps=1e-6, dtype=BF16, ws=None, wsb=0)
        return call(lib.block_norm_bwd, a, kw)

    for f in (block, block_back):
        assert f(x=None) == 1 and f(h=None) == 1 and f(groups=2) == 1 and f(s=FAKE) == 1 and f(s=FAKE, groups=4) == 1
        assert f(C=60) == 2 and f(C=8200) == 2 and f(rows=1 << 40) == 2 and f(rows=-1) == 1 and f(x=FAKE + 2) == 3
    assert block(rows=0) == 0 and block_back() == 4
    assert lib.block_norm_bwd_workspace_bytes(6, 64, 4) == BAD and lib.block_norm_bwd_workspace_bytes(6, 64, 3) not in (0, BAD)


def test_binding_refuses_host_tensors(lib):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(TypeError):
        binding.causal_conv_fwd(x, w)
    with pytest.raises(TypeError):
        binding.causal_conv_step(x[0], w, torch.zeros(4, 3, 8))
    with pytest.raises(TypeError):
        binding.ssm_scan_fwd(x, x, torch.zeros(8, 8), x, x)
    with pytest.raises(TypeError):
        binding.ssm_step(x[0], x[0], torch.zeros(8, 8), x[0], x[0], torch.zeros(4, 8, 8))
    with pytest.raises(TypeError):
        binding.gated_norm_fwd(x[None], x[None])
    with pytest.raises(TypeError):
        binding.block_norm_fwd(x, x)
