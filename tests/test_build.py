"""What the build makes: libraries that stay together when they are moved
(no GPU needed)."""

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
