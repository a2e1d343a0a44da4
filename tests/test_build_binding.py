"""The build of the Python extension (host compiler; no GPU): for which Python
and torch it was made, and what its failure leaves."""
import os
import sysconfig

import pytest
import torch

import token_dispatch_grouped_softmax_gb300 as moe
from token_dispatch_grouped_softmax_gb300 import _build, _lib


def test_another_torch_or_python_builds_it_again(monkeypatch):
    """An extension of another torch or Python is not taken for this one's."""
    moe.build()
    assert _build.up_to_date()
    assert os.path.samefile(_lib.binding().__file__, _build.binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0+none")
        assert not _build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".another-abi.so")
        assert not _build.up_to_date()
    assert _build.up_to_date()


def test_a_failed_extension_leaves_the_library(monkeypatch, tmp_path):
    """libmoe_gb300.so needs no torch and no host compiler's headers: it is
    linked all the same, and build() says what failed."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(_build, "sources", lambda: [str(src)])
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "ext.so"))
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "ext.so").exists()
