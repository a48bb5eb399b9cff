"""The windowed and 4-bit-cache forms through the index-checked build (libtva_checked.so):
they match float64 with no check firing, and an internal wait that runs out in the 4-bit
form's kernel ends in TVA_ERR_TIMEOUT with the context usable."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_matches_float64_with_no_check_firing():
    import __graft_entry__
    __graft_entry__.build()
    from tree_verification_attention_gb300 import build
    env = dict(os.environ, TVA_LIBRARY=build.CHECKED_LIB_PATH)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_checked_window_run.py")], env=env,
                       capture_output=True, text=True, timeout=900)
    print(r.stdout)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build: PASS" in r.stdout


@pytest.mark.parametrize("nodes", [[8], [64]])  # one and two row tiles a group
@pytest.mark.parametrize("kv4", [False, True])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_library_usable(nodes, kv4):
    from tests import _window
    from tree_verification_attention_gb300 import api
    pr = _window.Problem("bf16", [900], nodes, (32, 8), 128, "random", seed=50, kv4=kv4)
    t = pr.device()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.diag_set_wait_limit(5_000_000, True)   # 5 ms, and a wait that nothing completes
    try:
        pr.call(t, 300, 4, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 6
    finally:
        api.diag_set_wait_limit()
    out, lse = pr.run(300, 4, t)
    pr.check(out, lse, 300, 4)
