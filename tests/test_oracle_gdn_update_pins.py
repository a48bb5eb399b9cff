"""Pins of the Gated DeltaNet update and commit oracles."""
import numpy as np
import pytest

import oracle
from tree_verification_attention_gb300 import workloads


def _case(lens, heads=2, d=8, seed=1):
    pars = [workloads.chain_tree(n) for n in lens]
    return workloads.make_gdn_case(batch=len(lens), heads=heads, d=d, seed=seed, parents=pars)


def test_a_sequence_of_tokens_is_a_chain_of_the_tree():
    c = _case([5, 1, 9])
    out, _ = oracle.gdn_update(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["cu_nodes"], c["S0"])
    ref = oracle.gdn_tree_outputs(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["S0"], c["parent"], c["cu_nodes"])
    assert np.abs(out - ref).max() < 1e-12


def test_the_closed_product_form():
    """S_n = (prod_t A_t) S_0 + sum_t (prod_{s > t} A_s) b_t, A_t = alpha_t (I - beta_t k k^T)."""
    c = _case([6], heads=1)
    _, S = oracle.gdn_update(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["cu_nodes"], c["S0"])
    k, v, be, al = (c[n][:, 0].astype(np.float64) for n in ("k", "v", "beta", "alpha"))
    A = [al[t] * (np.eye(8) - be[t] * np.outer(k[t], k[t])) for t in range(6)]
    total = np.linalg.multi_dot(A[::-1]) @ c["S0"][0, 0]
    for t in range(6):
        P = np.eye(8)
        for s in range(t + 1, 6):
            P = A[s] @ P
        total = total + P @ (be[t] * np.outer(k[t], v[t]))
    assert np.abs(S[0, 0] - total).max() < 1e-12


@pytest.mark.parametrize("cut", [0, 1, 4, 7])
def test_a_prompt_in_two_parts_is_the_prompt(cut):
    c = _case([7])
    a = {n: c[n] for n in ("q", "k", "v", "beta", "alpha")}
    out, S = oracle.gdn_update(**a, cu_tokens=[0, 7], state=c["S0"])
    o1, S1 = oracle.gdn_update(**{n: x[:cut] for n, x in a.items()}, cu_tokens=[0, cut], state=c["S0"])
    o2, S2 = oracle.gdn_update(**{n: x[cut:] for n, x in a.items()}, cu_tokens=[0, 7 - cut], state=S1)
    assert np.abs(np.concatenate([o1, o2]) - out).max() < 1e-12 and np.abs(S2 - S).max() < 1e-12


def test_associative_recall_and_decay():
    """alpha = beta = 1, orthonormal keys: the state holds v_j under k_j; a later write under the same
    key replaces it; alpha = 0 forgets everything before."""
    k = np.eye(4)[[0, 1, 0]][:, None, :]
    v = np.arange(12.0).reshape(3, 1, 4)
    one = np.ones((3, 1))
    _, S = oracle.gdn_update(k, k, v, one, one, [0, 3], np.zeros((1, 1, 4, 4)))
    assert np.array_equal(S[0, 0], np.stack([v[2, 0], v[1, 0], np.zeros(4), np.zeros(4)]))
    gone = one.copy()
    gone[2] = 0.0
    _, S = oracle.gdn_update(k, k, v, one, gone, [0, 3], np.full((1, 1, 4, 4), 3.0))
    assert np.array_equal(S[0, 0], np.outer(k[2, 0], v[2, 0]))


def test_the_commit_is_the_update_over_the_path_and_what_the_tree_read():
    c = workloads.make_gdn_case(batch=2, heads=2, d=8, m=12, tree="random", seed=3)
    par, cu = c["parent"], c["cu_nodes"]
    path = []
    for b in range(2):
        j, up = 11 - b, []
        while j >= 0:
            up.append(j)
            j = int(par[cu[b] + j])
        path.append(up[::-1])
    lens = [len(p) for p in path]
    flat = np.concatenate([p + [-1] * (12 - len(p)) for p in path])
    S = oracle.commit_accepted_gdn(cu, lens, flat, c["k"], c["v"], c["beta"], c["alpha"], c["S0"])
    tree = oracle.gdn_tree_outputs(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["S0"], par, cu)
    for b in range(2):
        last = int(cu[b]) + path[b][-1]
        for h in range(2):  # the committed state read by the last node's query: that node's output
            assert np.abs(S[b, h].T @ c["q"][last, h] - tree[last, h]).max() < 1e-12
    none = oracle.commit_accepted_gdn(cu, [0, 0], flat, c["k"], c["v"], c["beta"], c["alpha"], c["S0"])
    assert np.array_equal(none, c["S0"])
