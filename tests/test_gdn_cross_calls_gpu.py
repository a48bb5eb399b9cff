"""Calls of the Gated DeltaNet state operators and of cross-attention as programs make them: prompts in
several segments, graphs, streams, kept workspaces, empty batches, waits that run out, refusals."""
import pytest
import torch

from tests import _gdn
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu

SEGMENTS = [  # more sequences and heads than one segment takes: 8 chunks (512 tokens) at a time
    (64, 16, 64, [1100, 0, 513] + [30] * 61),
    (32, 32, 128, [530, 1, 1025, 512] + [0] * 27 + [600]),
    (32, 32, 128, [900] + [3] * 30 + [0]),          # the launch's last block has no tokens
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield
    api.diag_set_wait_limit(0, False)


def _rows(t):
    return [t[n] for n in ("q", "k", "v", "beta", "alpha")]


def _reference(t, cu):
    """The recurrence in float64, heads and sequences side by side."""
    lens = [cu[i + 1] - cu[i] for i in range(len(cu) - 1)]
    S = t["state"].double().clone()
    out = torch.zeros(t["v"].shape, dtype=torch.float64, device="cuda")
    first = torch.tensor(cu[:-1], device="cuda")
    for step in range(max(lens)):
        live = torch.tensor([b for b, n in enumerate(lens) if n > step], device="cuda")
        at = first[live] + step
        k, v, q = (t[n][at].double() for n in ("k", "v", "q"))
        a, be = t["alpha"][at].double()[..., None], t["beta"][at].double()[..., None]
        w = be * (v - a * torch.einsum("bhkv,bhk->bhv", S[live], k))
        S[live] = a[..., None] * S[live] + k[..., None] * w[..., None, :]
        out[at] = torch.einsum("bhkv,bhk->bhv", S[live], q)
    return out, S


@pytest.mark.parametrize("which", range(len(SEGMENTS)))
def test_prompts_of_several_segments(which):
    B, H, d, lens = SEGMENTS[which]
    c = _gdn.case(lens, heads=H, d=d, dtype="bf16", seed=60 + which)
    t = _gdn.device(c, "bf16")
    assert api.gdn_workspace_size(B, H, d, torch.bfloat16, sum(lens), max(lens)) > api.gdn_workspace_size(
        B, H, d, torch.bfloat16, sum(lens), 512)
    out, S = _gdn.run(t, max(lens))
    ref, S_ref = _reference(t, c["cu_nodes"].tolist())
    _gdn.check(out, S, ref, S_ref, "bf16", max(lens))
    again = _gdn.run(t, max(lens))
    assert torch.equal(out, again[0]) and torch.equal(S, again[1])


def test_several_segments_captured_and_replayed_with_a_kept_workspace():
    B, H, d, lens = SEGMENTS[0]
    t = _gdn.device(_gdn.case(lens, heads=H, d=d, dtype="bf16", seed=70), "bf16")
    ws = torch.empty(api.gdn_workspace_size(B, H, d, torch.bfloat16, sum(lens), max(lens)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    S, S2, out = t["state"].clone(), t["state"].clone(), torch.empty_like(t["v"])
    api.gdn_update_varlen(*_rows(t), t["cu_tokens"], max(lens), S.clone(), workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):   # two calls after another, in one workspace
            api.gdn_update_varlen(*_rows(t), t["cu_tokens"], max(lens), S, out=out, dev_status=st, workspace=ws)
    for _ in range(3):
        g.replay()
        for _ in range(2):
            ref = api.gdn_update_varlen(*_rows(t), t["cu_tokens"], max(lens), S2)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(S, S2) and int(st.item()) == 0


def test_back_to_back_steps_on_one_stream():
    """Prompt, 40 single tokens, commits between them, without a wait: the same as with one after each."""
    H, d, B = 8, 128, 6
    lens = [100, 65, 1, 200, 33, 64]
    t = _gdn.device(_gdn.case(lens, heads=H, d=d, dtype="bf16", seed=71), "bf16")
    x = _gdn.device(_gdn.case([40] * B, heads=H, d=d, dtype="bf16", seed=72), "bf16")
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    length = torch.ones(B, dtype=torch.int32, device="cuda")
    path = torch.zeros(B, dtype=torch.int32, device="cuda")
    ends = []
    for wait in (True, False):
        S, outs = t["state"].clone(), []
        outs.append(api.gdn_update_varlen(*_rows(t), t["cu_tokens"], max(lens), S))
        for i in range(40):
            pick = torch.arange(i, 40 * B, 40, device="cuda")
            row = [y[pick].contiguous() for y in _rows(x)]
            if i % 3 == 2:
                api.commit_accepted_gdn(one, length, path, *row[1:], S, max_nodes=1)
            else:
                outs.append(api.gdn_update_varlen(*row, one, 1, S))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        ends.append((S, torch.cat(outs)))
    assert torch.equal(ends[0][0], ends[1][0]) and torch.equal(ends[0][1], ends[1][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_tokens_at_all(dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.empty(0, 2, 64, device="cuda", dtype=dt)
    g = torch.empty(0, 2, device="cuda")
    S = torch.randn(3, 2, 64, 64, device="cuda")
    before, cu, st = S.clone(), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for most in (0, 500):
        assert api.gdn_update_varlen(q, q, q, g, g, cu, most, S, dev_status=st).shape == (0, 2, 64)
    api.commit_accepted_gdn(cu, torch.zeros(3, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                            q, q, g, g, S, max_nodes=4, dev_status=st)
    torch.cuda.synchronize()
    assert torch.equal(S, before) and int(st.item()) == 0


@pytest.mark.parametrize("d,lens", [(128, [300, 64]), (64, [200])])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_library_usable(d, lens):
    c = _gdn.case(lens, heads=3, d=d, dtype="bf16", seed=73)
    t = _gdn.device(c, "bf16")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    S = t["state"].clone()
    api.diag_set_wait_limit(5_000_000, True)   # 5 ms, and a wait that nothing completes
    try:
        api.gdn_update_varlen(*_rows(t), t["cu_tokens"], max(lens), S, dev_status=st)
        torch.cuda.synchronize()
    finally:
        api.diag_set_wait_limit()
    assert int(st.item()) == 6 and torch.equal(S, t["state"])
    out, S = _gdn.run(t, max(lens))
    ref, S_ref = _gdn.recurrence(*_rows(t), c["cu_nodes"], t["state"])
    _gdn.check(out, S, ref, S_ref, "bf16", max(lens))


def test_a_status_word_made_on_another_stream_keeps_what_the_kernel_reports():
    """The current stream is busy; the call's own allocations belong to the stream it runs on."""
    side = torch.cuda.Stream()
    c = _gdn.case([100], heads=2, d=64, dtype="bf16", seed=74)
    t = _gdn.device(c, "bf16")
    S = t["state"].clone()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    bad = api.commit_accepted_gdn(cu, torch.full((1,), 2, dtype=torch.int32, device="cuda"),
                                  torch.zeros(100, dtype=torch.int32, device="cuda"), *_rows(t)[1:], S, max_nodes=4,
                                  stream=side)
    out = api.gdn_update_varlen(*_rows(t), t["cu_tokens"], 100, S, stream=side)
    torch.cuda.synchronize()
    assert int(bad.item()) == 1
    ref, S_ref = _gdn.recurrence(*_rows(t), c["cu_nodes"], t["state"])
    _gdn.check(out, S, ref, S_ref, "bf16", 100)


def test_refusals_of_the_binding():
    t = _gdn.device(_gdn.case([50, 3], heads=2, d=64, dtype="bf16", seed=75), "bf16")
    q, k, v, be, al = _rows(t)
    S, cu = t["state"], t["cu_tokens"]
    wrong = [
        (q.float(), k, v, be, al, cu, 50, S), (q, k, v, be.double(), al, cu, 50, S), (q, k, v, be, al, cu.long(), 50, S),
        (q, k, v, be, al, cu, 50, S.bfloat16()), (q, k, v, be, al, cu, 50, S[:1]), (q, k, v[:, :1], be, al, cu, 50, S),
        (q[:, :, ::2], k, v, be, al, cu, 50, S), (q, k, v, be[:50], al, cu, 50, S), (q, k, v, be, al, cu, 2 ** 31, S),
        (q, k, v, be, al, cu, 1.5, S), (q, k, v, be, al, cu, 50, S.transpose(2, 3)), (q, k, v, be, al, cu[:1], 50, S[:0]),
    ]
    for args in wrong:
        with pytest.raises(ValueError):
            api.gdn_update_varlen(*args)
    for out in (torch.empty_like(v).float(), v[:5], torch.empty(53, 2, 128, device="cuda", dtype=v.dtype)[:, :, ::2]):
        with pytest.raises(ValueError):
            api.gdn_update_varlen(q, k, v, be, al, cu, 50, S, out=out)
    for kw in (dict(out=v), dict(out=q), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(api.TvaError):
            api.gdn_update_varlen(q, k, v, be, al, cu, 50, S, **kw)
    both = torch.zeros(S.numel() + v.numel(), device="cuda")   # v's rows in the state's memory
    S2 = both[: S.numel()].view(S.shape)
    v2 = both[S.numel() - 64:].view(torch.bfloat16)[: v.numel()].view(v.shape)
    with pytest.raises(api.TvaError):
        api.gdn_update_varlen(q, k, v2, be, al, cu, 50, S2)
    with pytest.raises(api.TvaError):
        api.commit_accepted_gdn(cu, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                torch.zeros(53, dtype=torch.int32, device="cuda"), k, v2, be, al, S2, max_nodes=50)
    i = torch.zeros(53, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.commit_accepted_gdn(cu, i[:1], i, k, v, be, al, S)
    with pytest.raises(ValueError):
        api.commit_accepted_gdn(cu, i[:2], i[:9], k, v, be, al, S)
    with pytest.raises(api.TvaError):
        api.commit_accepted_gdn(cu, i[:2], i, k, v, be, al, S, max_nodes=129)

