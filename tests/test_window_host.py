"""The windowed walk of the attention kernels (which tiles are read, which keys of them a
row sees), compiled for the host and compared with the definition key by key
(tests/window_host.cpp)."""
import os
import shutil
import subprocess

import pytest

from tests.test_schedule_host import HERE, _cuda_include
from tree_verification_attention_gb300 import build


def test_windowed_walk_is_the_definition(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    inc = _cuda_include()
    if cxx is None or inc is None:
        pytest.skip("needs a C++ compiler and the CUDA headers")
    exe = str(tmp_path / "window_host")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I" + inc, "-I" + build.CSRC, "-I" + build.INCLUDE,
                    os.path.join(HERE, "window_host.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 2000
