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
