"""Problems and tolerances for the windowed and 4-bit-cache attention tests."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from tree_verification_attention_gb300 import api

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def tree(rng, kind, m):
    if kind == "chain":
        return np.arange(-1, m - 1, dtype=np.int32)
    if kind == "roots":
        return np.full(m, -1, dtype=np.int32)
    return np.array([-1 if i == 0 else int(rng.integers(-1, i)) for i in range(m)], dtype=np.int32)


class Problem:
    """Host tensors of one ragged batch; ``values`` gives the float64 values that the
    library is given (K / V of the cache from its records when ``kv4``)."""

    def __init__(self, dtype, prefixes, nodes, heads=(8, 2), d=64, kind="random", seed=0, kv4=False, spare=3,
                 spread=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed + 1)
        self.dtype, self.d, self.kv4 = dtype, d, kv4
        self.hq, self.hkv = heads
        dt = DTYPES[dtype]
        self.cu_prefix = np.concatenate([[0], np.cumsum(prefixes)]).astype(np.int32)
        self.cu_nodes = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.parent = np.concatenate([tree(rng, kind, m) for m in nodes]).astype(np.int32)
        self.max_prefix, self.max_nodes = max(prefixes), max(1, max(nodes))
        N, R = int(sum(nodes)), int(sum(prefixes)) + spare
        draw = lambda n, h: torch.randn(n, h, d, generator=gen)  # noqa: E731
        self.q = (spread * draw(N, self.hq)).to(dt)
        self.tree_k, self.tree_v = draw(N, self.hkv).to(dt), draw(N, self.hkv).to(dt)
        self.k, self.v = draw(R, self.hkv).to(dt), draw(R, self.hkv).to(dt)
        if kv4:
            self.records = torch.from_numpy(oracle.kv4_pack(self.k.double().numpy(), self.v.double().numpy()))

    def cache_values(self):
        if self.kv4:
            return oracle.kv4_values(self.records.numpy(), self.d)
        return self.k.double().numpy(), self.v.double().numpy()

    def reference(self, window, sinks):
        k, v = self.cache_values()
        return oracle.tree_verify_window_attention(
            self.q.double().numpy(), k, v, self.cu_prefix, self.tree_k.double().numpy(), self.tree_v.double().numpy(),
            self.parent, self.cu_nodes, self.hkv, window, sinks)

    def device(self):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        t = dict(q=self.q.cuda(), tree_k=self.tree_k.cuda(), tree_v=self.tree_v.cuda(), parent=i32(self.parent),
                 cu_prefix=i32(self.cu_prefix), cu_nodes=i32(self.cu_nodes))
        if self.kv4:
            t["kv4_cache"] = self.records.cuda()
        else:
            t["k_cache"], t["v_cache"] = self.k.cuda(), self.v.cuda()
        return t

    def call(self, t, window, sinks, **more):
        tail = (t["tree_k"], t["tree_v"], t["parent"], t["cu_prefix"], t["cu_nodes"], self.max_prefix, self.max_nodes)
        if self.kv4:
            return api.tree_verify_attn_kv4_varlen(t["q"], t["kv4_cache"], *tail, window=window, sinks=sinks, **more)
        return api.tree_verify_attn_window_varlen(t["q"], t["k_cache"], t["v_cache"], *tail, window=window, sinks=sinks,
                                                  **more)

    def run(self, window, sinks, t=None):
        t = t or self.device()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = self.call(t, window, sinks, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return out, lse

    def check(self, out, lse, window, sinks, where=""):
        """Against float64, at the errors that the arithmetic allows.

        A logit is a sum of d products in fp32 (each of its d + 2 operations off by at
        most 2^-24 of sum |q_i k_i|, at most Z) and passes through a base-2 scaling and
        subtraction (2^-22 of its size): e = (d + 8) 2^-24 Z with Z = max |q| |k| scale.
        Weights are then off by 2 e relative (itself and the sum), plus 2^-22 of the
        exponential and (n + 8) 2^-24 for n additions; for 16-bit inputs they are rounded
        once (half a step u), fp16 ones below 2^-14 by up to 2^-25 of the largest weight's
        2^8 at most.  The output is rounded once more (u of its size)."""
        ref, L, weight = self.reference(window, sinks)
        u = HALF_STEP[self.dtype]
        k, v = self.cache_values()
        n = self.max_prefix + self.max_nodes
        norm = lambda x: np.sqrt(np.nanmax((np.where(np.isfinite(x), x, 0) ** 2).sum(-1)))  # noqa: E731
        Z = norm(self.q.double().numpy()) * max(norm(k), norm(self.tree_k.double().numpy())) / np.sqrt(self.d)
        e = (self.d + 8) * 2.0 ** -24 * Z
        rel = 2 * e + 2.0 ** -22 + (n + 8) * 2.0 ** -24 + (0.0 if self.dtype == "fp32" else u)
        tol = rel * weight + u * np.abs(ref) + 1e-7
        if self.dtype == "fp16":
            tol = tol + n * 2.0 ** -25 * max(np.abs(np.where(np.isfinite(v), v, 0)).max(), 5.0)
        got = out.double().cpu().numpy()
        err = np.abs(got - ref)
        assert np.isfinite(got).all(), where
        assert (err <= tol).all(), (where, float((err / tol).max()), float(err.max()))
        lerr = np.abs(lse.double().cpu().numpy() - L)
        ltol = 2 * e + 2.0 ** -21 + (n + 8) * 2.0 ** -24 + 2.0 ** -21 * np.abs(L)
        assert (lerr <= ltol).all(), (where, float(lerr.max()))
