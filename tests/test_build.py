"""What the build makes: libraries that stay together when they are moved, and
a binding that is built again for another torch (no GPU needed)."""

import os
import shutil
import subprocess
import sys

from sparse_dictionary_coded_b200 import build

_MOVED = """
import sys
sys.path.insert(0, sys.argv[1])
import sparse_dictionary_coded_b200 as sdk
sdk._load_binding()
print(sorted({line.split()[-1] for line in open("/proc/self/maps") if "libsdk.so" in line}))
"""


def test_a_moved_package_uses_its_own_library(tmp_path):
    """The binding of a copy of the package calls the copy's library."""
    name = os.path.basename(build.PKG)
    shutil.copytree(build.PKG, tmp_path / name, ignore=shutil.ignore_patterns("csrc", "__pycache__"))
    r = subprocess.run([sys.executable, "-c", _MOVED, str(tmp_path)], cwd=str(tmp_path),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str([str(tmp_path / name / "libsdk.so")])


def test_binding_is_built_again_for_another_torch(tmp_path, monkeypatch):
    src, out, of = (tmp_path / n for n in ("binding.cpp", "_binding.so", "binding.of"))
    monkeypatch.setattr(build, "BINDING", str(out))
    monkeypatch.setattr(build, "BINDING_OF", str(of))
    src.write_text("")
    assert build.binding_stale(str(src), "python 3, torch 2.11")
    out.write_text("")
    assert build.binding_stale(str(src), "python 3, torch 2.11")      # built for what?
    of.write_text("python 3, torch 2.11")
    assert not build.binding_stale(str(src), "python 3, torch 2.11")
    assert build.binding_stale(str(src), "python 3, torch 2.12")
    os.utime(out, (0, 0))
    assert build.binding_stale(str(src), "python 3, torch 2.11")
