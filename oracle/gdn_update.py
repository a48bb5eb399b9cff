"""A Gated DeltaNet layer's tokens, and the commit of an accepted path into its state.

TEST INFRASTRUCTURE ONLY (see the package docstring): never called by the library.

The update is that of :mod:`oracle.gdn_tree` ("DFlash-TfM", Method 3), run token by token:
    S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t.
The page defers the tree's state update until the accepted branch is known; the commit is the
same recurrence over the accepted nodes, root first.
"""
from __future__ import annotations

import numpy as np

from .gdn_tree import gdn_path_state

__all__ = ["gdn_update", "commit_accepted_gdn"]


def gdn_update(q, k, v, beta, alpha, cu_tokens, state):
    """(o [n, H, dv], new state [B, H, dk, dv]) in float64.

    q, k [n, H, dk]; v [n, H, dv]; beta, alpha [n, H]; cu_tokens [B+1]; state [B, H, dk, dv]."""
    q = np.asarray(q, dtype=np.float64)
    S = np.array(state, dtype=np.float64, copy=True)
    out = np.zeros(np.asarray(v).shape)
    cu = np.asarray(cu_tokens, dtype=np.int64)
    for b in range(len(cu) - 1):
        for t in range(int(cu[b]), int(cu[b + 1])):
            for h in range(q.shape[1]):
                S[b, h] = gdn_path_state(S[b, h], k[:, h], v[:, h], beta[:, h], alpha[:, h], [t])
                out[t, h] = S[b, h].T @ q[t, h]
    return out, S


def commit_accepted_gdn(cu_nodes, accept_len, accept_path, k, v, beta, alpha, state):
    """The new state [B, H, dk, dv] after each sequence's accepted nodes (local ids)."""
    S = np.array(state, dtype=np.float64, copy=True)
    for b in range(len(accept_len)):
        n0 = int(cu_nodes[b])
        path = [n0 + int(p) for p in accept_path[n0:n0 + int(accept_len[b])]]
        for h in range(S.shape[1]):
            S[b, h] = gdn_path_state(S[b, h], k[:, h], v[:, h], beta[:, h], alpha[:, h], path)
    return S
