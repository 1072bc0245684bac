"""The layer operators' native module: only they need it, and it is taken for
the torch and Python that it was built for alone."""
import os

import pytest
import torch

from gated_delta_rule_47_gb300 import binding, build


@pytest.fixture
def unloaded(monkeypatch):
    """The binding as it is before its first call."""
    build.build()
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_front", None)
    return monkeypatch


def test_other_operators_do_without_it(unloaded):
    unloaded.setattr(binding, "FRONT_PATH", os.path.join(build.OUT_DIR, "absent.so"))
    assert binding.load().gdn_status_string(0) == b"GDN_OK"
    assert isinstance(binding.workspace_bytes(1, 2, 300, 64, 64, dtype=torch.float32), int)
    with pytest.raises(RuntimeError, match="absent.so"):  # and not the long way, slower and unseen
        binding.rms_norm_fwd(torch.zeros(2, 64))


def test_loaded_by_the_first_call(unloaded):
    binding.load()
    assert binding._front is None
    with pytest.raises(TypeError):
        binding.rms_norm_fwd(torch.zeros(2, 64))
    assert binding._front is not None


def test_built_for_this_torch(unloaded):
    assert binding.FRONT_PATH == build.front_path(torch.__version__) and os.path.exists(binding.FRONT_PATH)
    assert build.front_path("1.0") != build.front_path("1.1")  # one built before an upgrade is not found after it
