"""What build.py compiles, and when (CPU only; the compilers are stand-ins)."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "block_text_diffusion_b200")


@pytest.fixture
def tree(tmp_path):
    """The sources in a folder of their own, and a stand-in for nvcc that writes its -o file."""
    pkg = tmp_path / "pkg"
    shutil.copytree(os.path.join(PACKAGE, "csrc"), pkg / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copy(os.path.join(PACKAGE, "build.py"), pkg / "build.py")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text("#!/bin/sh\nwhile [ \"$1\" != -o ]; do shift; done\necho library > \"$2\"\n")
    nvcc.chmod(0o755)
    return tmp_path


def test_the_library_builds_without_torch(tree):
    code = ("import sys; sys.modules['torch'] = None; sys.path.insert(0, sys.argv[1]); import build; "
            "print(build.build())")
    r = subprocess.run([sys.executable, "-c", code, str(tree / "pkg")], capture_output=True, text=True,
                       env=dict(os.environ, NVCC=str(tree / "nvcc")))
    assert r.returncode == 0, r.stderr
    assert (tree / "pkg" / "libdg.so").read_text() == "library\n"
    assert not (tree / "pkg" / "_serving.so").exists() and "torch is not installed" in r.stderr


def load(tree, monkeypatch):
    spec = importlib.util.spec_from_file_location("build_in_a_tree", tree / "pkg" / "build.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    calls = []

    def compile_(cmd):
        calls.append(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binding")

    monkeypatch.setattr(module.subprocess, "check_call", compile_)
    return module, calls


def test_the_binding_is_rebuilt_for_another_torch_or_python(tree, monkeypatch):
    pytest.importorskip("torch")
    b, calls = load(tree, monkeypatch)
    b.build_binding()
    b.build_binding()
    assert calls == ["g++"] and b.binding_built_for() == b.binding_key()
    key = b.binding_key()
    monkeypatch.setattr(b, "binding_key", lambda: key.replace("torch ", "torch 9"))
    b.build_binding()
    b.build_binding()
    assert calls == ["g++"] * 2
    os.remove(b.BINDING_KEY)   # a binding of unknown origin
    b.build_binding()
    assert calls == ["g++"] * 3
    late = os.path.getmtime(b.BINDING) + 5
    os.utime(b.BINDING_SOURCES[0], (late, late))
    b.build_binding()
    assert calls == ["g++"] * 4


def test_nothing_is_needed_where_all_is_built(tree, monkeypatch):
    pytest.importorskip("torch")
    b, calls = load(tree, monkeypatch)
    monkeypatch.setenv("NVCC", str(tree / "nvcc"))
    lacks = b.binding_lacks
    monkeypatch.setattr(b, "binding_lacks", lambda: "")   # (the stand-in has no headers beside it)
    b.build()
    assert calls == [str(tree / "nvcc"), "g++"]

    def missing():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(b, "nvcc", missing)
    monkeypatch.setattr(b, "binding_lacks", lacks)
    assert b.build() == b.LIB and len(calls) == 2
    os.remove(b.BINDING)
    assert b.build() == b.LIB and len(calls) == 2   # a binding that cannot be compiled is no error


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    from block_text_diffusion_b200 import build, serving
    build.build()
    monkeypatch.setattr(serving, "_bound", None)
    serving._native()
    monkeypatch.setattr(serving, "_bound", None)
    monkeypatch.setattr(build, "binding_key", lambda: "torch 0.0\n")
    with pytest.raises(RuntimeError, match="another torch"):
        serving._native()
