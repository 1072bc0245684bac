"""Outputs whose elements share memory are refused at the C interface: two
threads would write one place.  Nothing here reaches a kernel."""
import ctypes

import pytest

from gated_delta_rule_47_gb300 import binding, build
from tests.test_layer_abi import bwd, fwd

INVALID, WORKSPACE = 1, 4  # without a workspace a call that passes its checks ends with the latter


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def strides(**kw):
    """Of contiguous q, k [1,1,8,64], v, o [1,2,8,64], g [1,2,8], but for those given."""
    a = dict(q=(0, 512, 64), k=(0, 512, 64), v=(0, 512, 64), o=(0, 512, 64), g=(0, 8, 1))
    a.update(kw)
    return (ctypes.c_longlong * 15)(*(x for n in ("q", "k", "v", "o", "g") for x in a[n]))


APART = [{}, dict(v=(0, 64, 128), o=(0, 64, 128), g=(0, 1, 2)), dict(q=(0, 0, 200), k=(0, 8, 72)), dict(v=(7 * 8, 1024, 128)),
         dict(o=(0, 64, 256), g=(5, 40, 5))]


@pytest.mark.parametrize("st", APART)
def test_apart(lib, st):
    assert fwd(lib, st=strides(**st)) == WORKSPACE and bwd(lib, st=strides(**st)) == WORKSPACE


@pytest.mark.parametrize("st", [dict(o=(0, 512, 0)), dict(o=(0, 64, 64)), dict(o=(0, 0, 64)), dict(o=(0, 128, 32))])
def test_forward(lib, st):
    assert fwd(lib, st=strides(**st)) == INVALID


@pytest.mark.parametrize("st", [dict(q=(0, 0, 0)), dict(k=(0, 0, 56)), dict(v=(0, 0, 64)), dict(v=(0, 256, 64)), dict(g=(0, 0, 1)),
                                dict(g=(0, 8, 0)), dict(g=(0, 1, 1))])
def test_backward(lib, st):
    assert bwd(lib, st=strides(**st)) == INVALID
    assert fwd(lib, st=strides(**st)) == WORKSPACE  # reading them is fine
