"""Cross-attention onto a cache of another length: one softmax per (query, head) over all of
the sequence's keys.

TEST INFRASTRUCTURE ONLY (see the package docstring): never called by the library.

LongSpec ("Memory-Efficient Architecture"): the draft layer's cross-attention reads the target
model's K/V cache.  No mask applies and the queries bring no keys.  Readings: contiguous query
head groups (head h reads KV head h / (Hq / Hkv)) and scale 1/sqrt(d), as for the tree; a
query without any key has output 0 and log-sum-exp -inf (an empty sum).
"""
from __future__ import annotations

import numpy as np

__all__ = ["cross_attention"]


def cross_attention(q, k_cache, v_cache, cu_queries, cu_keys, num_kv_heads, scale=None):
    """(out [N, Hq, d], lse [N, Hq]) in float64."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k_cache, v_cache))
    N, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros((N, Hq, d)), np.full((N, Hq), -np.inf)
    for b in range(len(cu_keys) - 1):
        p0, p1 = int(cu_keys[b]), int(cu_keys[b + 1])
        for i in range(int(cu_queries[b]), int(cu_queries[b + 1])):
            for h in range(Hq if p1 > p0 else 0):
                g = h // (Hq // num_kv_heads)
                z = scale * (k[p0:p1, g] @ q[i, h])
                w = np.exp(z - z.max())
                out[i, h] = w @ v[p0:p1, g] / w.sum()
                lse[i, h] = z.max() + np.log(w.sum())
    return out, lse
