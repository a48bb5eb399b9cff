"""The windowed and 4-bit-cache calls on a stream that is not the current one, and index
arrays that do not belong together."""
import pytest
import torch

from tests import _window
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _busy():
    torch.cuda._sleep(20_000_000)  # about 10 ms of the current stream


def test_a_status_word_made_by_the_call_keeps_what_the_kernel_reports():
    """The current stream is busy: a word zeroed there would be zeroed after the kernel on
    the other stream has written it."""
    side = torch.cuda.Stream()
    cache = api.alloc_kv4_cache(8, 2, 64)
    k = torch.randn(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    slot = torch.tensor([0, 8, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    _busy()
    st = api.append_kv4(k, k, slot, cache, stream=side)
    torch.cuda.synchronize()
    assert int(st.item()) == 1
    cu, one = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda")
    path, dst = torch.tensor([5, 0, 0], dtype=torch.int32, device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    _busy()
    st = api.commit_accepted_kv4(cu, one, path, k, k, dst, cache, max_nodes=3, stream=side)
    torch.cuda.synchronize()
    assert int(st.item()) == 1


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("positional", [False, True])
def test_a_call_on_another_stream_allocates_there(kv4, positional, monkeypatch):
    """What the call allocates and lets go of must belong to the stream that still uses it."""
    pr = _window.Problem("bf16", [700, 33], [9, 4], (8, 2), 128, "random", seed=3, kv4=kv4)
    t = pr.device()
    side = torch.cuda.Stream()
    seen = []
    alloc = api.alloc_workspace

    def spy(p, device):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return alloc(p, device)

    monkeypatch.setattr(api, "alloc_workspace", spy)
    torch.cuda.synchronize()
    _busy()
    cache = [t["kv4_cache"]] if kv4 else [t["k_cache"], t["v_cache"]]
    call = api.tree_verify_attn_kv4_varlen if kv4 else api.tree_verify_attn_window_varlen
    head = [t["q"], *cache, t["tree_k"], t["tree_v"], t["parent"], t["cu_prefix"], t["cu_nodes"], pr.max_prefix,
            pr.max_nodes, 64, 4]
    if positional:
        out, lse = call(*head, None, None, None, None, 0.0, side)
    else:
        out, lse = call(*head, stream=side)
    side.synchronize()
    assert seen == [side.cuda_stream]
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream
    pr.check(out, lse, 64, 4)
    if kv4:
        torch.cuda.synchronize()
        k, v = api.read_kv4(t["kv4_cache"], 128, stream=side)
        side.synchronize()
        again = api.read_kv4(t["kv4_cache"], 128)
        assert torch.equal(k, again[0]) and torch.equal(v, again[1])


@pytest.mark.parametrize("kv4", [False, True])
def test_index_arrays_of_different_batches_are_refused(kv4):
    pr = _window.Problem("bf16", [40, 33], [3, 4], (8, 2), 64, "random", seed=4, kv4=kv4)
    t = pr.device()
    for bad in (dict(cu_nodes=t["cu_nodes"][:2]), dict(cu_prefix=t["cu_prefix"][:2]),
                dict(cu_prefix=t["cu_prefix"][None], cu_nodes=t["cu_nodes"][None])):
        with pytest.raises(ValueError):
            pr.call(dict(t, **bad), 64, 4)
