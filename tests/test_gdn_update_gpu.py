"""Gated DeltaNet tokens (gdn_update_varlen) and the commit of an accepted path
(commit_accepted_gdn) against float64 (bars: tests/_gdn.py)."""
import numpy as np
import pytest
import torch

import oracle
from tests import _gdn
from tree_verification_attention_gb300 import api, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


LENGTHS = [
    [1], [2], [7], [8], [9], [16], [17], [63], [64], [65], [127], [128], [129], [200],
    [0, 1, 0], [1, 1, 1, 1, 1], [3, 0, 70, 64, 1], [130, 5, 33], [16, 2, 9], [0, 0],
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", range(len(LENGTHS)))
def test_against_the_definition(which, d, dtype):
    lens = LENGTHS[which]
    c = _gdn.case(lens, heads=1 + which % 3, d=d, dtype=dtype, seed=100 + which)
    out, S = _gdn.run(_gdn.device(c, dtype), max(lens))
    ref, S_ref = oracle.gdn_update(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["cu_nodes"], c["S0"])
    _gdn.check(out, S, ref, S_ref, dtype, max(lens))


@pytest.mark.parametrize("dtype,d,heads,lens", [
    ("bf16", 128, 5, [1000]), ("bf16", 64, 3, [777, 1, 2049]), ("fp32", 128, 3, [701, 64]),
    ("bf16", 128, 40, [100] * 9), ("bf16", 128, 32, [1] * 70), ("bf16", 64, 16, [65, 3] * 20), ("fp32", 64, 7, [40] * 33),
])
def test_longer_runs_and_larger_batches(dtype, d, heads, lens):
    c = _gdn.case(lens, heads=heads, d=d, dtype=dtype, seed=len(lens))
    t = _gdn.device(c, dtype)
    out, S = _gdn.run(t, max(lens))
    ref, S_ref = _gdn.recurrence(*(t[n] for n in ("q", "k", "v", "beta", "alpha")), c["cu_nodes"], t["state"])
    _gdn.check(out, S, ref, S_ref, dtype, max(lens))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[3, 1], [100, 65]])
def test_decays_of_zero_and_one_no_writes_and_full_writes(dtype, lens):
    """alpha = 0 forgets everything before, 1 nothing; beta 0 writes nothing, 1 replaces."""
    c = _gdn.case(lens, heads=4, d=128, dtype=dtype, seed=9)
    rng = np.random.default_rng(4)
    c["alpha"][:, 0], c["alpha"][:, 1] = 1.0, rng.choice([0.0, 1.0, 0.5], c["alpha"].shape[0])
    c["alpha"][:, 2] = rng.choice([1e-30, 1.0, 1e-4], c["alpha"].shape[0])
    c["beta"][:, 0], c["beta"][:, 3] = rng.choice([0.0, 1.0], c["beta"].shape[0]), 1.0
    t = _gdn.device(c, dtype)
    out, S = _gdn.run(t, max(lens))
    ref, S_ref = _gdn.recurrence(*(t[n] for n in ("q", "k", "v", "beta", "alpha")), c["cu_nodes"], t["state"])
    _gdn.check(out, S, ref, S_ref, dtype, max(lens))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_repeated_keys(dtype):
    """Every token under one of two keys: the triangular systems are as full as they get."""
    c = _gdn.case([150], heads=2, d=128, dtype=dtype, seed=10)
    c["k"][:] = c["k"][np.random.default_rng(1).integers(0, 2, 150)]
    c["beta"][:] = 0.98
    c["alpha"][:] = 0.999
    t = _gdn.device(c, dtype)
    out, S = _gdn.run(t, 150)
    ref, S_ref = _gdn.recurrence(*(t[n] for n in ("q", "k", "v", "beta", "alpha")), c["cu_nodes"], t["state"])
    _gdn.check(out, S, ref, S_ref, dtype, 150)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,most", [([2, 0, 5], 5), ([70, 0, 64, 3], 70), ([2, 0, 5], 100)])
def test_what_no_token_touches_stays(dtype, lens, most):
    """Rows behind the last sequence hold NaN and are neither read nor written; a sequence without
    tokens keeps its state bit for bit."""
    c = _gdn.case(lens, heads=2, d=64, dtype=dtype, seed=11)
    t = _gdn.device(c, dtype, spare=150)
    n = sum(lens)
    mark = torch.full_like(t["v"], 7.0)
    out, S = _gdn.run(t, most, out=mark)
    assert out is mark and (out[n:] == 7.0).all()
    ref, S_ref = oracle.gdn_update(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["cu_nodes"], c["S0"])
    _gdn.check(out, S, ref, S_ref, dtype, most)
    assert torch.equal(S[1], t["state"][1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_neighbour_s_rows_do_not_leak(dtype):
    """A sequence of NaN between two others spoils itself alone."""
    lens = [70, 66, 65]
    c = _gdn.case(lens, heads=2, d=128, dtype=dtype, seed=12)
    for n in ("q", "k", "v"):
        c[n][70:136] = np.nan
    t = _gdn.device(c, dtype)
    out, S = _gdn.run(t, 70)
    for b, (lo, hi) in enumerate([(0, 70), (70, 136), (136, 201)]):
        if b == 1:
            assert torch.isnan(S[1]).any()
            continue
        part = [t[n][lo:hi] for n in ("q", "k", "v", "beta", "alpha")]
        ref, S_ref = _gdn.recurrence(*part, [0, hi - lo], t["state"][b:b + 1])
        _gdn.check(out[lo:hi], S[b:b + 1], ref, S_ref, dtype, 70)


@pytest.mark.parametrize("most", [5, 100])
def test_bad_bounds_are_reported_and_skipped(most):
    """A sequence longer than max_tokens, or beyond the rows, keeps its state; the others run."""
    c = _gdn.case([3, 4, 2], heads=2, d=64, dtype="bf16", seed=13)
    t = _gdn.device(c, "bf16")
    t["cu_tokens"] = torch.tensor([0, 3, 7, 200], dtype=torch.int32, device="cuda")
    mark = torch.full_like(t["v"], 7.0)
    out, S = _gdn.run(t, most, out=mark, status=1)
    assert torch.equal(S[2], t["state"][2]) and (out[7:] == 7.0).all()
    part = [t[n][:7] for n in ("q", "k", "v", "beta", "alpha")]
    ref, S_ref = _gdn.recurrence(*part, [0, 3, 7], t["state"][:2])
    _gdn.check(out[:7], S[:2], ref, S_ref, "bf16", most)
    t["cu_tokens"] = torch.tensor([-2, 1, 1, 1], dtype=torch.int32, device="cuda")
    mark.fill_(7.0)
    out, S = _gdn.run(t, most, out=mark, status=1)
    assert torch.equal(S, t["state"]) and (out == 7.0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_prompt_in_parts_is_the_prompt(dtype):
    c = _gdn.case([300], heads=3, d=128, dtype=dtype, seed=14)
    t = _gdn.device(c, dtype)
    ref, S_ref = _gdn.recurrence(*(t[n] for n in ("q", "k", "v", "beta", "alpha")), [0, 300], t["state"])
    S, outs = t["state"].clone(), []
    for lo, hi in ((0, 64), (64, 65), (65, 81), (81, 300)):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        outs.append(api.gdn_update_varlen(*(t[n][lo:hi] for n in ("q", "k", "v", "beta", "alpha")), cu, hi - lo, S))
    _gdn.check(torch.cat(outs), S, ref, S_ref, dtype, 300)


def test_the_same_call_twice_gives_the_same_bits():
    for lens in ([1] * 9, [200, 77]):
        t = _gdn.device(_gdn.case(lens, heads=4, d=128, dtype="bf16", seed=15), "bf16")
        a, b = _gdn.run(t, max(lens)), _gdn.run(t, max(lens))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens", [[1, 1, 1], [150, 40, 64]])
def test_captured_and_replayed(lens):
    t = _gdn.device(_gdn.case(lens, heads=4, d=128, dtype="bf16", seed=16), "bf16")
    args = [t[n] for n in ("q", "k", "v", "beta", "alpha", "cu_tokens")]
    S, S2 = t["state"].clone(), t["state"].clone()
    out, st = torch.empty_like(t["v"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.gdn_update_varlen(*args, max(lens), S2.clone(), out=out, dev_status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.gdn_update_varlen(*args, max(lens), S, out=out, dev_status=st)
    for _ in range(3):
        g.replay()
        ref = api.gdn_update_varlen(*args, max(lens), S2)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(S, S2) and int(st.item()) == 0


def test_two_streams_at_once_and_a_stream_that_is_not_current():
    lens = [[300, 10], [129, 65]]
    ts = [_gdn.device(_gdn.case(n, heads=4, d=128, dtype="bf16", seed=17 + i), "bf16") for i, n in enumerate(lens)]
    alone = [_gdn.run(t, max(n)) for t, n in zip(ts, lens)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for t, n, s in zip(ts, lens, streams):
            S = t["state"].clone()
            s.wait_stream(torch.cuda.current_stream())
            got.append((api.gdn_update_varlen(*(t[x] for x in ("q", "k", "v", "beta", "alpha", "cu_tokens")), max(n), S,
                                              stream=s), S))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------ the commit

def _paths(c, seed, lens=None):
    """Root-to-node paths of the case's trees, or paths of the given lengths."""
    rng = np.random.default_rng(seed)
    cu, par = c["cu_nodes"], c["parent"]
    length, path = [], []
    for b in range(len(cu) - 1):
        m = int(cu[b + 1] - cu[b])
        up, j = [], int(rng.integers(0, m)) if m else -1
        while j >= 0:
            up.append(j)
            j = int(par[cu[b] + j])
        up = up[::-1][:None if lens is None else lens[b]]
        length.append(len(up))
        path += up + [-1] * (m - len(up))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(length), i32(path)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree,m,batch", [("chain", 128, 2), ("random", 40, 5), ("random", 1, 3), ("best_first", 64, 3)])
def test_commit_against_the_definition(tree, m, batch, d, dtype):
    c = workloads.make_gdn_case(batch=batch, heads=3, d=d, m=m, tree=tree, seed=m + batch, dtype=dtype)
    t = _gdn.device(c, dtype)
    for lens in (None, [1] * batch, [0, 3] + [0] * (batch - 2)):
        length, path = _paths(c, 5, lens)
        S = t["state"].clone()
        st = api.commit_accepted_gdn(t["cu_tokens"], length, path, t["k"], t["v"], t["beta"], t["alpha"], S)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        S_ref = oracle.commit_accepted_gdn(c["cu_nodes"], length.tolist(), path.tolist(), c["k"], c["v"], c["beta"],
                                           c["alpha"], c["S0"])
        none = torch.zeros(0)
        _gdn.check(none, S, none, S_ref, dtype, 1)
        for b, n in enumerate(length.tolist()):
            if n == 0:
                assert torch.equal(S[b], t["state"][b])


def test_commit_reports_bad_paths_and_leaves_their_states():
    c = workloads.make_gdn_case(batch=4, heads=2, d=64, m=6, tree="chain", seed=3)
    t = _gdn.device(c, "fp32")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    path = [0, 1, 2, -1, -1, -1] * 4
    path[6 + 1] = 6      # sequence 1: an id past its nodes
    path[12 + 2] = -1    # sequence 2: an id missing
    for length, bad in (([3, 3, 3, 7], (1, 2, 3)), ([2, 1, 3, -1], (2, 3))):
        S = t["state"].clone()
        st = api.commit_accepted_gdn(t["cu_tokens"], i32(length), i32(path), t["k"], t["v"], t["beta"], t["alpha"], S,
                                     max_nodes=6)
        torch.cuda.synchronize()
        assert int(st.item()) == 1
        for b in range(4):
            assert torch.equal(S[b], t["state"][b]) == (b in bad), b
    S = t["state"].clone()
    st = api.commit_accepted_gdn(t["cu_tokens"], i32([1] * 4), i32(path), t["k"], t["v"], t["beta"], t["alpha"], S, max_nodes=5)
    torch.cuda.synchronize()
    assert int(st.item()) == 1 and torch.equal(S, t["state"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_speculative_cycle(dtype):
    """Prompt, draft tree, verification, the walk, the commit, one more token: the outputs and the
    state are those of the tokens run one after the other."""
    rng = np.random.default_rng(21)
    lens, B, H, d = [150, 64, 7], 3, 2, 128
    c = _gdn.case(lens, heads=H, d=d, dtype=dtype, seed=22)
    t = _gdn.device(c, dtype)
    state = torch.zeros(B, H, d, d, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.gdn_update_varlen(*(t[n] for n in ("q", "k", "v", "beta", "alpha", "cu_tokens")), max(lens), state, dev_status=st)
    tree = workloads.make_gdn_case(batch=B, heads=H, d=d, m=20, tree="random", seed=23, dtype=dtype)
    w = _gdn.device(tree, dtype)
    parent = torch.from_numpy(tree["parent"]).int().cuda()
    out = api.gdn_tree_verify(w["cu_tokens"], parent, w["q"], w["k"], w["v"], w["beta"], w["alpha"], state, max_nodes=20,
                              dev_status=st)
    tok = torch.from_numpy(rng.integers(0, 2, B * 20)).int().cuda()
    target = torch.from_numpy(rng.integers(0, 2, B * 21)).int().cuda()
    length, path, _ = api.accept_longest_path(w["cu_tokens"], parent, tok, target, dev_status=st)
    api.commit_accepted_gdn(w["cu_tokens"], length, path, w["k"], w["v"], w["beta"], w["alpha"], state, max_nodes=20,
                            dev_status=st)
    nxt = _gdn.case([1] * B, heads=H, d=d, dtype=dtype, seed=24)
    x = _gdn.device(nxt, dtype)
    last = api.gdn_update_varlen(*(x[n] for n in ("q", "k", "v", "beta", "alpha", "cu_tokens")), 1, state, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    first = 0
    for b, n in enumerate(lens):
        nodes = [b * 20 + p for p in path[b * 20:b * 20 + int(length[b])].tolist()]
        seq = {z: torch.cat([t[z][first:first + n], w[z][nodes], x[z][b:b + 1]]) for z in ("q", "k", "v", "beta", "alpha")}
        total = seq["k"].shape[0]
        ref, S_ref = _gdn.recurrence(**seq, cu=[0, total], state=torch.zeros(1, H, d, d, device="cuda"))
        got = torch.cat([out[nodes], last[b:b + 1]])
        _gdn.check(got, state[b:b + 1], ref[n:], S_ref, dtype, 1)
        first += n
