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
