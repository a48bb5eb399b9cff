"""The 4-bit-cache attention at every size of its row groups (few rows are computed by a
kernel of their own)."""
import pytest
import torch

from tests import _window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,m", [((4, 4), 1), ((2, 2), 31), ((2, 2), 32), ((2, 2), 33), ((8, 2), 8), ((8, 2), 9),
                                     ((8, 2), 16), ((8, 2), 17), ((3, 1), 10), ((3, 1), 11), ((3, 1), 21), ((3, 1), 22),
                                     ((32, 1), 1), ((32, 1), 2), ((64, 1), 1), ((65, 1), 1), ((5, 1), 25)])
def test_every_number_of_rows(dtype, d, heads, m):
    # prefixes that end inside each quarter of a tile, none at all, and many tiles a worker
    P = [0, 1, 31, 33, 70, 127, 128, 129, 20000 // (1 + m // 8)]
    pr = _window.Problem(dtype, P, [m] * len(P), heads, d, "random", seed=m, kv4=True)
    t = pr.device()
    for window, sinks in ((0, 0), (1, 0), (50, 4), (200, 130)):
        out, lse = pr.run(window, sinks, t)
        pr.check(out, lse, window, sinks, (window, sinks))
        again = pr.run(window, sinks, t)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("nodes", [[2, 0, 8, 1, 5, 8, 3], [16, 1, 0, 13], [1] * 70])
def test_trees_of_different_sizes_in_one_batch(nodes):
    P = [(937 * (b + 1)) % 1500 for b in range(len(nodes))]
    pr = _window.Problem("bf16", P, nodes, (32, 8), 128, "random", seed=len(nodes), kv4=True)
    t = pr.device()
    for window, sinks in ((0, 0), (300, 4)):
        out, lse = pr.run(window, sinks, t)
        pr.check(out, lse, window, sinks, (window, sinks))


def test_weights_that_differ_by_many_binades():
    """Logits of many sizes: the running maxima of a tile's parts differ, and move."""
    pr = _window.Problem("bf16", [1000], [4], (8, 2), 128, "chain", seed=9, kv4=True, spread=12.0)
    t = pr.device()
    out, lse = pr.run(0, 0, t)
    pr.check(out, lse, 0, 0)


def test_more_sequences_than_the_staged_arrays_hold():
    B = 600
    pr = _window.Problem("bf16", [(7 * b) % 300 for b in range(B)], [1] * B, (4, 1), 64, "chain", seed=21, kv4=True)
    t = pr.device()
    for window, sinks in ((0, 0), (100, 4)):
        out, lse = pr.run(window, sinks, t)
        pr.check(out, lse, window, sinks, (window, sinks))


def test_calls_on_two_streams_and_a_replayed_graph():
    """Two problems at once, each with its own workspace, then both captured and replayed."""
    prs = [_window.Problem("bf16", P, m, (32, 8), 128, "random", seed=31, kv4=True)
           for P, m in (([3000, 17, 900], [2, 1, 2]), ([5000], [4]))]
    ts = [pr.device() for pr in prs]
    streams = [torch.cuda.Stream() for _ in prs]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs = [pr.call(t, 0, 0, dev_status=st, stream=s) for pr, t, s in zip(prs, ts, streams)]
    torch.cuda.synchronize()
    for pr, (out, lse) in zip(prs, outs):
        pr.check(out, lse, 0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [pr.call(t, 0, 0, dev_status=st) for pr, t in zip(prs, ts)]
    for _ in range(3):
        for out, lse in held:
            out.zero_()
            lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for (out, lse), (o, l) in zip(held, outs):
            assert torch.equal(out, o) and torch.equal(lse, l)
    assert int(st.item()) == 0


def test_a_bad_tree_and_bad_lengths_are_reported():
    pr = _window.Problem("bf16", [300, 40], [3, 4], (8, 2), 128, "chain", seed=33, kv4=True)
    for name, at, value, code in (("parent", 4, 2, 3), ("parent", 1, -2, 3), ("cu_prefix", 2, 1 << 20, 1),
                                  ("cu_nodes", 1, 6, 1)):
        t = pr.device()
        t[name][at] = value
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        pr.call(t, 0, 0, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == code, (name, at)
