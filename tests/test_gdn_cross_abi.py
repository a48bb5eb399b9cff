"""Host-side refusals of the Gated DeltaNet state calls and of cross-attention (nothing is enqueued;
the pointers below are never dereferenced), and the tests' float64 recurrence against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import oracle
from tests import _gdn
from tree_verification_attention_gb300 import api

P = ctypes.c_void_p
A = 1 << 20
S = 1 << 30   # the state's fake address, O the output's
O = 1 << 32  # noqa: E741


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return api.load_library()


def test_the_tests_recurrence_is_the_oracle_s():
    c = _gdn.case([5, 0, 3], heads=2, d=64, seed=1)
    a = {n: torch.from_numpy(c[n]) for n in ("q", "k", "v", "beta", "alpha")}
    out, st = _gdn.recurrence(**a, cu=c["cu_nodes"], state=torch.from_numpy(c["S0"]))
    ref, S_ref = oracle.gdn_update(c["q"], c["k"], c["v"], c["beta"], c["alpha"], c["cu_nodes"], c["S0"])
    assert np.abs(out.numpy() - ref).max() < 1e-12 and np.abs(st.numpy() - S_ref).max() < 1e-12


def test_update_refusals(lib):
    def call(B=2, H=4, d=128, dtype=0, cap=64, most=32, cu=A, q=A, k=A, v=A, beta=A, alpha=A, state=S, out=O, ws=A,
             n=1 << 40, st=A):
        return lib.gdn_update_varlen(B, H, d, dtype, cap, most, P(cu), P(q), P(k), P(v), P(beta), P(alpha), P(state),
                                     P(out), P(ws), n, P(st), None)
    assert call(B=0) == 1 and call(H=0) == 1 and call(cap=-1) == 1 and call(most=-1) == 1
    assert call(cap=2 ** 31 - 1) == 1
    assert call(d=96) == 2 and call(dtype=2) == 2 and call(dtype=5) == 2
    for name in ("cu", "q", "k", "v", "beta", "alpha", "state", "out", "st"):
        assert call(**{name: None}) == 1, name
    for name, at in (("q", A), ("k", A), ("v", A), ("state", S), ("out", O)):
        assert call(**{name: at + 8}) == 1, name
    for name in ("q", "k", "v", "beta", "alpha", "out"):
        assert call(**{name: S + 64}) == 1, name       # inside the state
    for name in ("q", "k", "v", "beta", "alpha"):
        assert call(**{name: O + 64}) == 1, name       # inside the output
    assert call(B=1 << 13, H=1 << 12) == 1             # more states than a launch numbers
    need = lib.tva_gdn_workspace_size(2, 4, 128, 0, 64, 32)
    assert need > 0 and call(n=need - 1) == 4 and call(ws=None) == 4 and call(ws=A + 64) == 4


def test_workspace_sizes(lib):
    size = lib.tva_gdn_workspace_size
    assert size(1, 4, 128, 1, 100, 100) == 0 and size(64, 32, 128, 0, 64, 1) == 0 and size(1, 4, 96, 0, 64, 64) == 0
    assert size(0, 4, 128, 0, 64, 64) == 0 and size(1, 4, 128, 0, 64, 24) == 0 and size(1, 4, 64, 0, 64, 40) == 0
    assert size(1, 4, 128, 0, 8, 1 << 30) == 0                      # no more than 8 rows: the recurrence
    one = size(1, 1, 128, 0, 64, 64)
    assert one == size(1, 1, 128, 0, 64, 1 << 30) and size(2, 3, 128, 0, 1000, 128) == 12 * one
    assert size(64, 32, 128, 0, 1 << 20, 1 << 20) == 64 * 32 * 8 * 2 * one   # bounded, whatever the lengths


def test_commit_refusals(lib):
    def call(B=2, H=4, d=128, dtype=0, cap=64, most=32, cu=A, ln=A, path=A, k=A, v=A, beta=A, alpha=A, state=S, st=A):
        return lib.commit_accepted_gdn(B, H, d, dtype, cap, most, P(cu), P(ln), P(path), P(k), P(v), P(beta), P(alpha),
                                       P(state), P(st), None)
    assert call(B=0) == 1 and call(H=-1) == 1 and call(cap=-1) == 1 and call(most=0) == 1 and call(most=129) == 1
    assert call(d=32) == 2 and call(dtype=2) == 2
    for name in ("cu", "ln", "path", "k", "v", "beta", "alpha", "state", "st"):
        assert call(**{name: None}) == 1, name
    for name, at in (("k", A), ("v", A), ("state", S)):
        assert call(**{name: at + 4}) == 1, name
    assert call(k=S + 64) == 1 and call(alpha=S) == 1


def test_cross_refusals(lib):
    def params(**kw):
        base = dict(batch=1, num_q_heads=4, num_kv_heads=1, head_dim=64, dtype=0, softmax_scale=0.0, cu_prefix=8,
                    cu_nodes=8, max_prefix_len=256, max_nodes=8, kv_capacity=256, node_capacity=8)
        base.update(kw)
        return api.Params(**base)

    def call(p, q=A, k=A, v=A, out=A, lse=A, ws=A, n=1 << 40, st=A):
        return lib.cross_attn_varlen(ctypes.byref(p) if p else None, P(q), P(k), P(v), P(out), P(lse), P(ws), n, P(st), None)
    assert call(None) == 1
    for kw, code in ((dict(head_dim=96), 2), (dict(num_q_heads=6, num_kv_heads=4), 1), (dict(max_nodes=65537), 2),
                     (dict(max_nodes=0), 1), (dict(batch=0), 1), (dict(dtype=7), 2), (dict(max_prefix_len=-1), 1),
                     (dict(cu_nodes=None), 1), (dict(cu_prefix=None), 1), (dict(num_q_heads=258, num_kv_heads=2), 2)):
        assert call(params(**kw)) == code, kw
        if "cu_nodes" not in kw and "cu_prefix" not in kw:
            assert lib.tva_cross_workspace_size(ctypes.byref(params(**kw))) == 0
    ok = params()
    for name in ("q", "out"):
        assert call(ok, **{name: None}) == 1 and call(ok, **{name: A + 8}) == 1, name
    assert call(ok, lse=None) == 1 and call(ok, st=None) == 1 and call(ok, k=A + 8) == 1


def test_the_binding_refuses_host_tensors_and_bad_shapes():
    x, g, i = torch.zeros(4, 2, 64), torch.zeros(4, 2), torch.zeros(2, dtype=torch.int32)
    state = torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError):
        api.gdn_update_varlen(x, x, x, g, g, i, 4, state)
    with pytest.raises(ValueError):
        api.gdn_update_varlen(x, x, x, g, g, i, 1 << 40, state)
    with pytest.raises(ValueError):
        api.gdn_update_varlen(x.half(), x.half(), x.half(), g, g, i, 4, state)
    with pytest.raises(ValueError):
        api.commit_accepted_gdn(i, i[:1], i, x, x, g, g, state, max_nodes=4)
    with pytest.raises(ValueError):
        api.cross_attn_varlen(x, x, x, i, i, 4, 4)
    with pytest.raises(ValueError):
        api.cross_attn_varlen(x.double(), x, x, i, i, 4, 4)
