"""The windowed oracle against facts that fix it: the unwindowed oracle, banded causal
attention (torch, float64, explicit masks), keys listed one by one, and closed forms."""
import itertools

import numpy as np
import pytest
import torch

import oracle

D, HKV, G = 8, 2, 2


def _draw(rng, P, m):
    f = lambda n, h: rng.standard_normal((n, h, D))  # noqa: E731
    return f(m, HKV * G), f(P, HKV), f(P, HKV), f(m, HKV), f(m, HKV)


def _call(q, k, v, tk, tv, parent, P, window, sinks):
    return oracle.tree_verify_window_attention(q, k, v, [0, P], tk, tv, parent, [0, len(parent)], HKV, window, sinks)


@pytest.mark.parametrize("window", [0, 1000, 2 ** 31 - 1])
def test_a_window_longer_than_everything_changes_nothing(window):
    rng = np.random.default_rng(1)
    parent = [-1, 0, 0, 1, -1, 4]
    q, k, v, tk, tv = _draw(rng, 37, 6)
    out, lse, _ = _call(q, k, v, tk, tv, parent, 37, window, 3)
    ref, L = oracle.tree_verify_attention(q, k, v, [0, 37], tk, tv, np.asarray(parent), [0, 6], HKV)
    assert np.abs(out - ref).max() < 1e-13 and np.abs(lse - L).max() < 1e-13


@pytest.mark.parametrize("P,m,window,sinks", [(9, 4, 3, 0), (9, 4, 3, 2), (20, 12, 5, 4), (0, 7, 2, 0), (2, 7, 1, 4),
                                              (5, 3, 1, 0)])
def test_a_chain_is_banded_causal_attention(P, m, window, sinks):
    rng = np.random.default_rng(2)
    q, k, v, tk, tv = _draw(rng, P, m)
    out, _, _ = _call(q, k, v, tk, tv, np.arange(-1, m - 1), P, window, sinks)
    K = torch.from_numpy(np.concatenate([k, tk]).transpose(1, 0, 2)).repeat_interleave(G, 0)
    V = torch.from_numpy(np.concatenate([v, tv]).transpose(1, 0, 2)).repeat_interleave(G, 0)
    t, s = torch.arange(P, P + m)[:, None], torch.arange(P + m)[None, :]
    mask = (s <= t) & ((t - s < window) | (s < sinks))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q.transpose(1, 0, 2).copy()), K, V, mask)
    assert np.abs(out - ref.numpy().transpose(1, 0, 2)).max() < 1e-12


def test_every_small_tree_against_keys_listed_one_by_one():
    rng = np.random.default_rng(3)
    for m in (1, 2, 3, 4):
        for parent in itertools.product(*[range(-1, i) for i in range(m)]):
            for P, window, sinks in ((0, 1, 0), (3, 2, 1), (6, 3, 2), (6, 4, 0), (2, 2, 5)):
                q, k, v, tk, tv = _draw(rng, P, m)
                out, lse, _ = _call(q, k, v, tk, tv, parent, P, window, sinks)
                for n, h in itertools.product(range(m), range(HKV * G)):
                    o, L = oracle.tree_verify_window_rows(n, h, q, k, v, [0, P], tk, tv, parent, [0, m], HKV, window,
                                                          sinks)
                    assert np.abs(out[n, h] - o).max() < 1e-12 and abs(lse[n, h] - L) < 1e-12


def test_uniform_keys_count_the_visible_ones():
    P, window, sinks = 50, 10, 4
    parent = np.arange(-1, 15)
    q, k, v, tk, tv = (np.zeros(s) for s in ((16, HKV * G, D), (P, HKV, D), (P, HKV, D), (16, HKV, D), (16, HKV, D)))
    _, lse, _ = _call(q, k, v, tk, tv, parent, P, window, sinks)
    assert np.allclose(lse, np.log(window + sinks))


def test_rows_that_no_node_sees_are_not_touched():
    rng = np.random.default_rng(4)
    q, k, v, tk, tv = _draw(rng, 40, 3)
    k[4:31], v[4:31] = np.nan, np.inf
    out, lse, _ = _call(q, k, v, tk, tv, [-1, 0, 0], 40, 10, 4)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
