"""Windowed tree-verification attention against float64 on the GPU."""
import numpy as np
import pytest
import torch

from tests import _window
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


# (prefixes, nodes, heads, d, tree, window, sinks)
CASES = [
    ([300], [8], (8, 2), 64, "chain", 100, 4),
    ([0], [1], (4, 1), 64, "chain", 1, 0),                       # one node, no prefix
    ([1], [1], (4, 4), 128, "chain", 1, 0),                      # sees itself alone
    ([129], [1], (32, 8), 128, "chain", 128, 0),                 # a single token, prefix just out of reach
    ([1000], [1], (32, 8), 128, "chain", 512, 4),
    ([700], [128], (16, 2), 128, "chain", 5, 0),                 # windows shorter than the path; teams of workers
    ([700], [128], (16, 2), 128, "chain", 5, 130),               # deep rows: sinks alone
    ([900], [128], (64, 8), 128, "random", 300, 200),
    ([2000], [68], (32, 8), 128, "random", 1024, 0),
    ([513, 0, 127, 128, 129, 1], [9, 3, 1, 17, 2, 5], (8, 2), 64, "random", 128, 1),
    ([513, 0, 127, 128, 129, 1], [9, 3, 1, 17, 2, 5], (8, 2), 64, "random", 127, 128),
    ([300, 40, 260], [5, 0, 33], (12, 4), 128, "random", 33, 7),  # an empty tree between two others; G = 3
    ([300, 40, 260], [5, 0, 33], (12, 4), 64, "roots", 1, 300),
    ([640, 641, 5], [40, 40, 40], (32, 2), 128, "random", 260, 129),  # G = 16: several row groups
    ([600, 90], [100, 128], (4, 4), 64, "chain", 90, 3),
    ([500, 100], [7, 7], (8, 2), 128, "random", BIG, 4),          # a window longer than any position
    ([500, 100], [7, 7], (8, 2), 128, "random", 60, BIG),         # sinks: everything
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(dtype, case):
    P, m, heads, d, kind, window, sinks = CASES[case]
    pr = _window.Problem(dtype, P, m, heads, d, kind, seed=100 + case)
    out, lse = pr.run(window, sinks)
    pr.check(out, lse, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_random_shapes(dtype):
    rng = np.random.default_rng(8)
    for i in range(30):
        B = int(rng.integers(1, 12))
        P = [int(x) for x in rng.integers(0, 800, B)]
        m = [int(x) for x in rng.integers(0, 40, B)]
        m[0] = max(1, m[0])
        heads = [(4, 1), (8, 8), (16, 2), (12, 4), (6, 2)][int(rng.integers(5))]
        window, sinks = int(2 ** rng.uniform(0, 10)), int(rng.choice([0, 1, 4, 64, 131]))
        pr = _window.Problem(dtype, P, m, heads, int(rng.choice([64, 128])), str(rng.choice(["chain", "random"])), seed=i)
        out, lse = pr.run(window, sinks)
        pr.check(out, lse, window, sinks, (i, P, m, heads, window, sinks))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("nodes", [[3, 20], [40, 100]])  # one and two row tiles a group
def test_rows_that_no_node_sees_may_hold_anything(dtype, nodes):
    """Evicted rows, and rows behind the last sequence, hold NaN and infinities."""
    window, sinks = 70, 5
    pr = _window.Problem(dtype, [400, 333], nodes, (8, 2), 128, "random", seed=3, spare=200)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")]).to(pr.k.dtype)
    for b, P in enumerate((400, 333)):
        p0 = int(pr.cu_prefix[b])
        pr.k[p0 + sinks:p0 + P - window + 1] = bad[b]
        pr.v[p0 + sinks:p0 + P - window + 1] = bad[2 * b]
    pr.k[733:], pr.v[733:] = bad[0], bad[1]
    out, lse = pr.run(window, sinks)
    pr.check(out, lse, window, sinks)


def test_an_endless_window_is_the_unwindowed_call():
    pr = _window.Problem("bf16", [700, 0, 130], [30, 5, 1], (32, 8), 128, "random", seed=5)
    t = pr.device()
    out, lse = pr.run(BIG, 0, t)
    ref, rl = api.tree_verify_attn_varlen(t["q"], t["k_cache"], t["v_cache"], t["tree_k"], t["tree_v"], t["parent"],
                                          t["cu_prefix"], t["cu_nodes"], pr.max_prefix, pr.max_nodes)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_twice_the_same_and_rows_outside_are_left():
    """Two calls agree bit for bit; rows of out and lse past cu_nodes[B] are not written."""
    pr = _window.Problem("bf16", [700, 100], [30, 5], (32, 8), 128, "random", seed=6)
    t = pr.device()
    for k in ("q", "tree_k", "tree_v", "parent"):
        t[k] = torch.cat([t[k], t[k][:7]])
    outs = []
    for _ in range(2):
        out, lse = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:2], 7.0, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        pr.call(t, 200, 4, out=out, lse=lse, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and bool((out[35:] == 7).all()) and bool((lse[35:] == 7).all())
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    pr.check(outs[0][0][:35], outs[0][1][:35], 200, 4)


def test_a_captured_call_on_its_own_stream_replays_with_new_inputs():
    pr, other = (_window.Problem("bf16", [600, 200], [16, 9], (32, 8), 128, "chain", seed=s) for s in (7, 8))
    t, new = pr.device(), other.device()
    p = api.make_params(t["q"], t["k_cache"], t["cu_prefix"], t["cu_nodes"], 8, pr.max_prefix, pr.max_nodes)
    ws = api.alloc_workspace(p, "cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pr.call(t, 130, 4, out=out, lse=lse, workspace=ws, dev_status=st, params=p)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pr.call(t, 130, 4, out=out, lse=lse, workspace=ws, dev_status=st, params=p)
    for k in t:
        t[k].copy_(new[k])
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    other.check(out, lse, 130, 4)


def test_two_streams_with_workspaces_of_their_own():
    prs = [_window.Problem("bf16", [900, 50], [20, 3], (32, 8), 128, "random", seed=s) for s in (9, 10)]
    ts = [p.device() for p in prs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i] = prs[i].call(ts[i], 300, 4)
    torch.cuda.synchronize()
    for i in (0, 1):
        prs[i].check(*outs[i], 300, 4)


def test_device_errors_go_to_the_status_word():
    pr = _window.Problem("bf16", [300, 100], [6, 6], (8, 2), 64, "chain", seed=11)
    for key, value, code in (("parent", 5, 3), ("parent", -2, 3)):
        t = pr.device()
        t[key][2] = value
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        pr.call(t, 64, 4, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == code
    t = pr.device()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    small = api.make_params(t["q"], t["k_cache"], t["cu_prefix"], t["cu_nodes"], 2, 200, 6)  # max_prefix_len too small
    out, _ = pr.call(t, 64, 4, dev_status=st, params=small)
    torch.cuda.synchronize()
    assert int(st.item()) == 1


def test_the_binding_refuses_what_does_not_fit():
    pr = _window.Problem("bf16", [100], [4], (8, 2), 64, "chain", seed=12)
    t = pr.device()
    with pytest.raises(api.TvaError):
        pr.call(t, 0, 0)
    with pytest.raises(api.TvaError):
        pr.call(t, 8, -1)
    with pytest.raises(api.TvaError) as e:
        pr.call(t, 8, 0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
    for key in ("q", "k_cache", "tree_k"):
        strided = dict(t, **{key: torch.cat([t[key], t[key]], -1)[..., ::2]})
        with pytest.raises(ValueError):
            pr.call(strided, 8, 0)
    with pytest.raises(ValueError):
        pr.call(t, 8, 0, out=torch.empty(4, 8, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        pr.call(dict(t, k_cache=t["k_cache"].half()), 8, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("seed", range(6))
def test_batches_of_short_sequences_agree_call_after_call(dtype, seed):
    """Workers whose ranges cross several short row groups, in batches large enough for the
    staged running sums: right, and the same bits every time."""
    rng = np.random.default_rng(80 + seed)
    B = int(rng.integers(16, 48))
    P = [int(x) for x in rng.integers(0, (100, 300, 2000)[seed % 3], B)]
    m = [int(x) for x in rng.integers(0, 9 if seed % 2 else 50, B)]
    m[0] = 1
    heads, d = [((12, 4), 128), ((8, 2), 64), ((32, 8), 128)][seed % 3]
    window, sinks = (60, 4) if seed < 3 else (700, 0)
    pr = _window.Problem(dtype, P, m, heads, d, "random", seed=seed)
    t = pr.device()
    out, lse = pr.run(window, sinks, t)
    pr.check(out, lse, window, sinks, (B, P, m))
    for _ in range(10):
        again = pr.run(window, sinks, t)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_batches_beyond_the_staged_arrays():
    """Batches whose arrays no longer fit in shared memory, or whose sums do not."""
    for B in (200, 300, 700):
        rng = np.random.default_rng(B)
        P = [int(x) for x in rng.integers(0, 60, B)]
        m = [int(x) for x in rng.integers(0, 3, B)]
        m[0] = 1
        for dtype in ("bf16", "fp32"):
            pr = _window.Problem(dtype, P, m, (4, 2), 64, "random", seed=B)
            out, lse = pr.run(25, 3)
            pr.check(out, lse, 25, 3)
        pr = _window.Problem("bf16", P, m, (4, 2), 64, "random", seed=B, kv4=True)
        out, lse = pr.run(0, 0)
        pr.check(out, lse, 0, 0)
