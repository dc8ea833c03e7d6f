"""What the build makes and when it makes it again (compilers replaced by
stand-ins that only write their output files)."""

import os

import pytest

from weight_quantized_moe_gb300 import build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """build() into a folder of its own; returns the commands that ran."""
    ran = []

    def run(cmd, what, verbose=False):
        ran.append(what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoeq.so"))
    monkeypatch.setattr(build, "PYEXT", str(tmp_path / "_mx_binding.so"))
    return ran


def test_library_is_linked_where_the_binding_cannot_be_compiled(sandbox, monkeypatch):
    """Without torch's or Python's headers or a C++ compiler the C library is
    there all the same; the build says what failed."""
    def no_compiler():
        raise RuntimeError("g++ not found")
    monkeypatch.setattr(build, "_cxx", no_compiler)
    with pytest.raises(RuntimeError, match="g\\+\\+ not found"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.PYEXT)
    first = len(sandbox)
    with pytest.raises(RuntimeError, match="g\\+\\+ not found"):
        build.build()
    assert len(sandbox) == first        # the library is up to date: not compiled again


def test_build_makes_both_once(sandbox):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.PYEXT)
    assert build.up_to_date()
    first = len(sandbox)
    build.build()
    assert len(sandbox) == first


def test_binding_is_made_again_for_another_torch(sandbox, monkeypatch):
    """A binding belongs to the torch (and Python) that it was compiled against."""
    import torch
    build.build()
    first = len(sandbox)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not build.up_to_date()
    build.build()
    assert build.up_to_date()
    again = sandbox[first:]
    assert again and all("binding" in what for what in again)   # the library stays
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-0.so")
    assert not build.up_to_date()
