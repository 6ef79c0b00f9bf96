"""The library and its Python module are built each for itself: a module that cannot
be compiled leaves the library built and in date, and is never loaded into another
torch or Python than it was built for.  (No compiler runs here.)"""

import os
import subprocess

import pytest

from w4a16_nvfp4_weight_gb300 import _lib, build_lib


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """build_lib over an empty folder, with compilers that note what they are given."""
    class fake:
        calls = []
        broken = ()

    def run(cmd, **kw):
        src = next((os.path.basename(c) for c in cmd if c.endswith((".cu", ".cpp"))), None)
        if src:
            fake.calls.append(src)
        if src in fake.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    fake.calls = []
    for name, path in (("BUILD", tmp_path), ("LIB", tmp_path / "lib.so"), ("BINDING", tmp_path / "binding.so")):
        monkeypatch.setattr(build_lib, name, str(path))
    monkeypatch.setattr(build_lib.subprocess, "run", run)
    return fake


def test_a_module_that_does_not_compile_leaves_the_library(fake):
    fake.broken = ("binding.cpp",)
    with pytest.warns(UserWarning, match="Python.h"):
        assert build_lib.build() == build_lib.LIB
    assert os.path.exists(build_lib.LIB) and build_lib.library_up_to_date() and not build_lib.up_to_date()
    assert len(fake.calls) == len(build_lib.sources()) + 1
    del fake.calls[:]
    with pytest.warns(UserWarning):
        build_lib.build()                                      # the module alone is tried again
    assert fake.calls == ["binding.cpp"]
    fake.broken = ()
    build_lib.build()
    assert build_lib.up_to_date()
    del fake.calls[:]
    build_lib.build()
    assert fake.calls == []
    os.utime(build_lib.BINDING, (0, 0))                        # older than its source, which does not compile
    fake.broken = ("binding.cpp",)
    with pytest.warns(UserWarning):
        build_lib.build()
    assert not os.path.exists(build_lib.BINDING) and build_lib.library_up_to_date()


def test_a_module_of_another_torch_is_rebuilt_and_not_loaded(fake, monkeypatch):
    build_lib.build()
    monkeypatch.setattr(build_lib, "_binding_abi", lambda: "torch 0.0 other")
    assert build_lib.library_up_to_date() and not build_lib.binding_up_to_date()
    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(_lib, "load", lambda *a, **kw: None)
    with pytest.raises(RuntimeError, match="was built for torch"):
        _lib.load_binding()
    del fake.calls[:]
    build_lib.build()
    assert fake.calls == ["binding.cpp"] and build_lib.up_to_date()


def test_a_library_that_does_not_compile_raises(fake):
    fake.broken = (os.path.basename(build_lib.sources()[0]),)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build_lib.build()
    assert not os.path.exists(build_lib.LIB)
