"""The index-checked build (libtva_checked.so) over Gated DeltaNet prompts and cross-attention: the
results match with the device status still zero, so no index that the kernels compute left its
bounds."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_matches_with_no_check_firing():
    import __graft_entry__
    __graft_entry__.build()
    from tree_verification_attention_gb300 import build
    env = dict(os.environ, TVA_LIBRARY=build.CHECKED_LIB_PATH)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_checked_gdn_cross_run.py")], env=env,
                       capture_output=True, text=True, timeout=900)
    print(r.stdout)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build: PASS" in r.stdout
