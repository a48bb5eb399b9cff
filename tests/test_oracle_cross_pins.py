"""Pins of the cross-attention oracle."""
import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("hq,hkv", [(4, 1), (6, 3), (2, 2)])
def test_against_the_library_attention_without_a_mask(hq, hkv):
    rng = np.random.default_rng(hq)
    cu_q, cu_k = [0, 3, 4], [0, 7, 12]
    q, k, v = rng.standard_normal((4, hq, 8)), rng.standard_normal((12, hkv, 8)), rng.standard_normal((12, hkv, 8))
    out, lse = oracle.cross_attention(q, k, v, cu_q, cu_k, hkv)
    for b in range(2):
        qs = torch.from_numpy(q[cu_q[b]:cu_q[b + 1]]).transpose(0, 1)
        ks, vs = (torch.from_numpy(x[cu_k[b]:cu_k[b + 1]]).transpose(0, 1).repeat_interleave(hq // hkv, 0) for x in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(qs, ks, vs).transpose(0, 1).numpy()
        assert np.abs(out[cu_q[b]:cu_q[b + 1]] - ref).max() < 1e-12
        l = torch.logsumexp(qs @ ks.transpose(1, 2) / 8 ** 0.5, -1).T.numpy()
        assert np.abs(lse[cu_q[b]:cu_q[b + 1]] - l).max() < 1e-12


def test_without_keys():
    out, lse = oracle.cross_attention(np.ones((3, 2, 8)), np.ones((4, 1, 8)), np.ones((4, 1, 8)), [0, 2, 3], [0, 0, 4], 1)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    assert np.allclose(out[2], 1) and np.allclose(lse[2], 8 ** 0.5 + np.log(4))


def test_it_is_the_tree_attention_s_prefix_part():
    """Merged with the tree keys' own part it gives the hybrid attention."""
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((2, 2, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    tk, tv = rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    o1, l1 = oracle.cross_attention(q, k, v, [0, 2], [0, 9], 1)
    o, l = oracle.tree_verify_attention(q, k, v, [0, 9], tk, tv, [-1, 0], [0, 2], 1)
    for i in range(2):
        for h in range(2):
            z = tk[:i + 1, 0] @ q[i, h] / 8 ** 0.5
            l2 = np.log(np.exp(z).sum())
            o2 = np.exp(z - l2) @ tv[:i + 1, 0]
            both = np.logaddexp(l1[i, h], l2)
            assert abs(both - l[i, h]) < 1e-12
            assert np.abs(o1[i, h] * np.exp(l1[i, h] - both) + o2 * np.exp(l2 - both) - o[i, h]).max() < 1e-12
