"""Runs windowed and 4-bit-cache calls through the library named by TVA_LIBRARY (the
index-checked build, libtva_checked.so) and compares them with float64.  Executed as a child
process by tests/test_checked_window_gpu.py; exits 1 on a mismatch or a non-zero status."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import oracle  # noqa: E402
from tests import _window  # noqa: E402
from tree_verification_attention_gb300 import api  # noqa: E402

CASES = [
    ([0], [1], (4, 1), 64, "chain", 1, 0),
    ([700], [128], (16, 2), 128, "chain", 5, 130),
    ([900], [128], (64, 8), 128, "random", 300, 200),
    ([513, 0, 127, 128, 129, 1], [9, 3, 1, 17, 2, 5], (8, 2), 64, "random", 128, 1),
    ([640, 641, 5], [40, 40, 40], (32, 2), 128, "random", 260, 129),
    ([90 * i for i in range(20)], [i % 7 for i in range(1, 21)], (12, 4), 128, "random", 100, 4),
    ([211 * i for i in range(20)], [i % 3 for i in range(1, 21)], (8, 2), 128, "random", 300, 140),  # up to 8 rows
    ([97 * i for i in range(18)], [i % 4 for i in range(1, 19)], (20, 4), 64, "random", 0x7fffffff, 4),  # up to 15
]


def main():
    lib = api.load_library()
    assert os.path.basename(lib._name) == "libtva_checked.so", lib._name
    bad = 0
    for i, (P, m, heads, d, kind, window, sinks) in enumerate(CASES):
        for dtype, kv4 in (("bf16", False), ("fp16", False), ("fp32", False), ("bf16", True), ("fp16", True)):
            pr = _window.Problem(dtype, P, m, heads, d, kind, seed=40 + i, kv4=kv4)
            for w, s in ((window, sinks), (0, 0)) if kv4 else ((window, sinks),):
                try:
                    pr.check(*pr.run(w, s), w, s)
                    ok = True
                except AssertionError as e:
                    ok = False
                    print("mismatch", str(e)[:200])
                print("ok  " if ok else "FAIL", dtype, kv4, P, m, heads, w, s, flush=True)
                bad += 0 if ok else 1
    k, v = torch.randn(2, 50, 3, 128).to(torch.bfloat16)
    cache = api.alloc_kv4_cache(64, 3, 128)
    st = api.append_kv4(k.cuda(), v.cuda(), torch.arange(63, 13, -1, dtype=torch.int32, device="cuda"), cache)
    rec = oracle.kv4_pack(k.double().numpy(), v.double().numpy())
    bad += 0 if int(st.item()) == 0 and np.array_equal(cache.cpu().numpy()[14:][::-1], rec) else 1
    print("checked build:", "PASS" if bad == 0 else f"{bad} FAILED")
    sys.exit(1 if bad else 0)


if __name__ == "__main__":
    main()
