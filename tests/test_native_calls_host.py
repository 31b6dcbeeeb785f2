"""The library without the binding's native calls (no GPU)."""
import os
import sys

import pytest
import torch

import selective_state_space_44_amd as ssm
from selective_state_space_44_amd import _build


def test_the_library_loads_without_the_native_calls(monkeypatch):
    """The scan, the decode step and the masked-matrix form need libssm.so alone;
    what takes the native calls says that they are missing."""
    monkeypatch.setattr(ssm, "_lib", None)
    monkeypatch.setattr(ssm, "_calls", None)
    monkeypatch.setitem(sys.modules, ssm.__name__ + "._calls", None)   # its import fails
    assert ssm.load_library().ssm_abi_version() > 0
    assert ssm.scan_workspace_bytes(1, 64, 64) >= 0
    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(OSError, match="native calls"):
        ssm.linear_attn(x, x, x, torch.zeros(2))
    with pytest.raises(OSError, match="native calls"):
        ssm.qk_norm_rotate(x, x, None, None)


def test_the_library_is_built_where_the_native_calls_are_not(monkeypatch, tmp_path):
    """A failure of theirs is raised when the library stands."""
    def fail(*a):
        raise RuntimeError("no headers")
    monkeypatch.setattr(_build, "build_calls", fail)
    monkeypatch.setattr(_build, "SOURCES", ["ssm_linattn_step.hip"])
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    out = tmp_path / "lib.so"
    with pytest.raises(RuntimeError, match="no headers"):
        _build.build(out=str(out))
    assert os.path.getsize(out) > 0
