"""Tree-verification attention under a sliding window with sinks, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring): never called by the library.

Definition followed
-------------------
:mod:`oracle.tree_attention`'s single softmax over the concatenated prefix and tree keys,
with one more condition on visibility.  Positions: prefix row s of a sequence stands at s;
a tree node stands at the prefix length plus its number of proper ancestors.  A node at
position t sees the key at position s (a prefix row, an ancestor, or itself) when
t - s < window or s < sinks.  LongSpec's draft model attends through a window of 512
("Memory-Efficient Architecture") and its Anchor-Offset Indices keep positions 0 .. 3 as
sinks; the pages give no formula.
"""
from __future__ import annotations

import numpy as np

from .tree_attention import ancestor_mask

__all__ = ["window_visible", "tree_verify_window_rows", "tree_verify_window_attention"]


def window_visible(parent_local, prefix_len: int, window: int, sinks: int) -> np.ndarray:
    """vis[i, s]: node i sees key s of the prefix rows followed by the tree nodes.
    ``window`` 0: no window."""
    anc = ancestor_mask(parent_local)
    m = len(anc)
    position = np.concatenate([np.arange(prefix_len), prefix_len + anc.sum(axis=1) - 1]).astype(np.int64)
    reach = np.concatenate([np.ones((m, prefix_len), dtype=bool), anc], axis=1)
    if window == 0:
        return reach
    t = position[prefix_len:, None]
    return reach & ((t - position[None, :] < window) | (position[None, :] < sinks))


def tree_verify_window_attention(q, k_cache, v_cache, cu_prefix, tree_k, tree_v, parent, cu_nodes,
                                 num_kv_heads: int, window: int, sinks: int, softmax_scale=None):
    """(out [N, Hq, d], lse [N, Hq], weight [N, Hq, d]): weight is sum_s p_s |v_s|, the size
    that errors of the weights are measured against.  Rows of the cache that no node sees
    are not touched (they may hold NaN)."""
    q = np.asarray(q, dtype=np.float64)
    N, Hq, d = q.shape
    Hkv = int(num_kv_heads)
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if softmax_scale is None else float(softmax_scale)
    out, lse, weight = np.zeros((N, Hq, d)), np.zeros((N, Hq)), np.zeros((N, Hq, d))
    for b in range(len(cu_prefix) - 1):
        p0, p1, n0, n1 = (int(x) for x in (cu_prefix[b], cu_prefix[b + 1], cu_nodes[b], cu_nodes[b + 1]))
        m, P = n1 - n0, p1 - p0
        if m == 0:
            continue
        vis = window_visible(np.asarray(parent[n0:n1]), P, window, sinks)
        used = np.flatnonzero(vis.any(axis=0))
        vis = np.repeat(vis[:, used], G, axis=0)
        pre, own = used[used < P] + p0, used[used >= P] - P + n0
        for g in range(Hkv):
            K = np.concatenate([np.asarray(k_cache[pre, g], np.float64), np.asarray(tree_k[own, g], np.float64)])
            V = np.concatenate([np.asarray(v_cache[pre, g], np.float64), np.asarray(tree_v[own, g], np.float64)])
            Z = scale * (q[n0:n1, g * G:(g + 1) * G].reshape(m * G, d) @ K.T)
            Z = np.where(vis, Z, -np.inf)
            top = Z.max(axis=1, keepdims=True)
            L = top[:, 0] + np.log(np.exp(Z - top).sum(axis=1))
            W = np.exp(Z - L[:, None])
            out[n0:n1, g * G:(g + 1) * G] = (W @ V).reshape(m, G, d)
            weight[n0:n1, g * G:(g + 1) * G] = (W @ np.abs(V)).reshape(m, G, d)
            lse[n0:n1, g * G:(g + 1) * G] = L.reshape(m, G)
    return out, lse, weight


def tree_verify_window_rows(n, h, q, k_cache, v_cache, cu_prefix, tree_k, tree_v, parent, cu_nodes,
                            num_kv_heads: int, window: int, sinks: int):
    """The same definition for one node n and query head h, its keys listed one by one."""
    b = int(np.searchsorted(np.asarray(cu_nodes), n, side="right") - 1)
    p0, P, n0 = int(cu_prefix[b]), int(cu_prefix[b + 1] - cu_prefix[b]), int(cu_nodes[b])
    d, g = q.shape[2], h // (q.shape[1] // num_kv_heads)
    path, j = [], n - n0
    while j >= 0:  # itself first
        path.append(j)
        j = int(parent[n0 + j])
    t = P + len(path) - 1
    z, vals = [], []
    for s in range(P):
        if window == 0 or t - s < window or s < sinks:
            z.append(float(k_cache[p0 + s, g].astype(np.float64) @ q[n, h].astype(np.float64)) / np.sqrt(d))
            vals.append(v_cache[p0 + s, g].astype(np.float64))
    for back, node in enumerate(path):
        if window == 0 or back < window or t - back < sinks:
            z.append(float(tree_k[n0 + node, g].astype(np.float64) @ q[n, h].astype(np.float64)) / np.sqrt(d))
            vals.append(tree_v[n0 + node, g].astype(np.float64))
    z = np.asarray(z)
    L = z.max() + np.log(np.exp(z - z.max()).sum())
    return np.exp(z - L) @ np.asarray(vals), L
