"""The compiled Python binding belongs to one PyTorch, one Python and one header: with another, it is built anew or
refused, never imported."""
import os
import sysconfig

import pytest
import torch

from deepseek_v4_moe_gb300 import _lib, build, dense


@pytest.fixture
def fresh(monkeypatch):
    """Built and up to date, and nothing loaded as far as the package knows."""
    _lib.load()
    assert not build._stale()
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(dense, "_n", None)
    return monkeypatch


def test_the_binding_that_fits_is_loaded(fresh):
    assert dense._native().block_norm and not build._stale()


def other_torch(mp, _):
    mp.setattr(torch, "__version__", "0.0.0+other")


def other_cuda(mp, _):
    mp.setattr(torch.version, "cuda", "0.0")


def other_python(mp, _):
    known = sysconfig.get_config_var
    mp.setattr(sysconfig, "get_config_var", lambda name: "cpython-00" if name in ("SOABI", "EXT_SUFFIX") else known(name))


def other_header(mp, tmp_path):
    path = tmp_path / "moe_ffn.h"
    path.write_text("/* another interface, older than what is built */\n")
    os.utime(path, (0, 0))
    mp.setattr(build, "INCLUDE", str(tmp_path))


@pytest.mark.parametrize("change", [other_torch, other_cuda, other_python, other_header])
def test_another_environment_is_another_binding(fresh, change, tmp_path):
    change(fresh, tmp_path)
    assert build._stale()


@pytest.mark.parametrize("change", [other_torch, other_python])
def test_a_binding_that_cannot_be_built_is_not_replaced_by_an_older_one(fresh, change, tmp_path):
    def fails(*a, **kw):
        raise RuntimeError("g++ failed on binding.cpp")

    change(fresh, tmp_path)
    fresh.setattr(build, "build", fails)
    with pytest.raises(RuntimeError) as e:
        dense._native()
    assert "_native" in str(e.value) and "g++ failed" in str(e.value.__cause__)
    assert dense._n is None
    _lib.load()  # the library itself, which knows nothing of PyTorch, stays usable
