"""The device-side timeout path of the windowed and the 4-bit-cache partials kernels: a wait
that nothing completes runs out (the library's diagnostic hook), the kernel lets the copies
it has started finish, frees its tensor memory and reports TVA_ERR_TIMEOUT, and the next
call on the same stream is right."""
import pytest
import torch

from tests import _window
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield
    api.diag_set_wait_limit(0, False)


@pytest.mark.parametrize("prefixes,nodes,heads,d", [([900], [6], (8, 2), 128), ([1500], [60], (32, 8), 128),
                                                    ([900], [100], (32, 4), 128), ([700, 0, 50], [20, 3, 33], (8, 2), 64)],
                         ids=["one M-tile", "two M-tiles", "shared teams", "batch d64"])
@pytest.mark.parametrize("kv4", [False, True])
def test_expired_wait_reports_timeout_and_the_next_call_is_right(kv4, prefixes, nodes, heads, d):
    pr = _window.Problem("bf16", prefixes, nodes, heads, d, "random", seed=5, kv4=kv4)
    t = pr.device()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        api.diag_set_wait_limit(50_000, True)  # 50 us, and a wait nothing completes
        pr.call(t, 300, 4, dev_status=st)
        torch.cuda.synchronize()
    finally:
        api.diag_set_wait_limit(0, False)
    assert int(st.item()) == 6
    out, lse = pr.run(300, 4, t)
    pr.check(out, lse, 300, 4)
