"""Runs Gated DeltaNet prompts and cross-attention through the library named by TVA_LIBRARY (the
index-checked build, libtva_checked.so) and compares them with float64.  Executed as a child process by
tests/test_checked_gdn_cross_gpu.py; exits 1 on a mismatch or a non-zero status."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from tests import _gdn, test_cross_gpu  # noqa: E402
from tree_verification_attention_gb300 import api  # noqa: E402


def main():
    lib = api.load_library()
    assert os.path.basename(lib._name) == "libtva_checked.so", lib._name
    bad = 0

    def run(what, call):
        nonlocal bad
        try:
            call()
            print("ok  ", what, flush=True)
        except AssertionError as e:
            bad += 1
            print("FAIL", what, str(e)[:200], flush=True)

    def update(dtype, d, lens):
        c = _gdn.case(lens, heads=3, d=d, dtype=dtype, seed=80)
        t = _gdn.device(c, dtype, spare=70)
        out, S = _gdn.run(t, max(lens))
        n = sum(lens)
        ref, S_ref = _gdn.recurrence(*(t[x][:n] for x in ("q", "k", "v", "beta", "alpha")), c["cu_nodes"], t["state"])
        _gdn.check(out, S, ref, S_ref, dtype, max(lens))

    for dtype in ("bf16", "fp32"):
        for d in (64, 128):
            for lens in ([64], [1, 0, 130], [65, 200, 64, 7]):
                run(("update", dtype, d, lens), lambda: update(dtype, d, lens))  # noqa: B023
    for i, (keys, queries, heads, d) in enumerate(test_cross_gpu.CASES):
        for dtype in ("bf16", "fp16", "fp32"):
            pr = test_cross_gpu.Problem(dtype, keys, queries, heads, d, seed=90 + i)
            run(("cross", dtype, keys[:4], queries[:4], heads, d), lambda: pr.check(*pr.run()))  # noqa: B023
    print("checked build:", "PASS" if bad == 0 else f"{bad} FAILED")
    sys.exit(1 if bad else 0)


if __name__ == "__main__":
    main()
