"""What the build makes: the C library on any machine with nvcc, the tensor module
where torch is installed, named by the torch and Python that it was built for.
The compilers are replaced by ones that only write their output file."""

import os
import subprocess
import sysconfig

import pytest

from speculative_decoding_tree_sv_gb300 import build


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    run.calls = calls
    return run


def test_the_library_builds_without_torch(compilers, monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    lib = build.build()
    assert os.path.exists(lib) and build.up_to_date() and build.marshal_path() is None
    assert all(cmd[0] == "nvcc" for cmd in compilers.calls)
    n = len(compilers.calls)
    assert build.build() == lib and len(compilers.calls) == n  # nothing left to do


def test_the_library_is_in_place_when_the_module_fails(compilers, monkeypatch):
    run = build.subprocess.run

    def no_module(cmd, **kw):
        if any(str(x).endswith("marshal.cpp") for x in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        return run(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", no_module)
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        build.build()
    assert os.path.exists(build.library_path()) and not build.up_to_date()


def test_another_torch_builds_its_own_module(compilers, monkeypatch):
    build.build()
    first = build.marshal_path()
    assert build.up_to_date() and os.path.exists(first) and first.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(build, "_torch_version", lambda where: "9.9.9")
    assert build.marshal_path() != first and not build.up_to_date()
    build.build()
    assert build.up_to_date() and os.path.exists(build.marshal_path()) and os.path.exists(first)


def test_the_module_is_named_by_the_torch_that_is_imported():
    import torch
    assert f"torch{torch.__version__}" in build.marshal_path()
