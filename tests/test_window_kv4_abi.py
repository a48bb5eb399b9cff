"""Host-side refusals of the windowed and 4-bit-cache entry points: an error code, and
nothing enqueued (the pointers below are never dereferenced)."""
import ctypes

import pytest
import torch

import __graft_entry__
from tree_verification_attention_gb300 import api

P = ctypes.c_void_p
A = 1 << 20  # fake, aligned addresses


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return api.load_library()


def _params(**kw):
    base = dict(batch=1, num_q_heads=4, num_kv_heads=1, head_dim=64, dtype=0, softmax_scale=0.0, cu_prefix=8,
                cu_nodes=8, max_prefix_len=256, max_nodes=8, kv_capacity=256, node_capacity=8)
    base.update(kw)
    return api.Params(**base)


def _window(lib, p, window=16, sinks=0, q=A, k=A, v=A, tk=A, tv=A, par=A, out=A, lse=A, ws=A, n=1 << 40, st=A):
    return lib.tree_verify_attn_window_varlen(ctypes.byref(p) if p else None, window, sinks, P(q), P(k), P(v), P(tk),
                                              P(tv), P(par), P(out), P(lse), P(ws), n, P(st), None)


def _kv4(lib, p, window=0, sinks=0, q=A, c=A, tk=A, tv=A, par=A, out=A, lse=A, ws=A, n=1 << 40, st=A):
    return lib.tree_verify_attn_kv4_varlen(ctypes.byref(p) if p else None, window, sinks, P(q), P(c), P(tk), P(tv),
                                           P(par), P(out), P(lse), P(ws), n, P(st), None)


@pytest.mark.parametrize("call", [_window, _kv4])
def test_attention_refusals(lib, call):
    ok = _params()
    assert call(lib, None) == 1
    assert call(lib, ok, window=-1) == 1 and call(lib, ok, sinks=-1) == 1
    if call is _window:
        assert call(lib, ok, window=0) == 1
    for kw, code in ((dict(head_dim=96), 2), (dict(num_q_heads=6, num_kv_heads=4), 1), (dict(max_nodes=129), 2),
                     (dict(batch=0), 1), (dict(dtype=7), 2), (dict(max_prefix_len=-1), 1), (dict(cu_nodes=None), 1),
                     (dict(num_q_heads=258, num_kv_heads=2), 2)):
        assert call(lib, _params(**kw)) == code, kw
    for name in ("q", "tk", "tv", "out"):
        assert call(lib, ok, **{name: None}) == 1 and call(lib, ok, **{name: A + 8}) == 1, name
    for name in ("par", "lse", "st"):
        assert call(lib, ok, **{name: None}) == 1, name
    assert call(lib, ok, **{"k" if call is _window else "c": None}) == 1
    assert call(lib, ok, **{"k" if call is _window else "c": A + 4}) == 1


def test_kv4_attention_refuses_fp32(lib):
    assert _kv4(lib, _params(dtype=1)) == 2


def test_record_bytes(lib):
    assert [lib.tva_kv4_record_bytes(d) for d in (64, 128, 96, 0, -64)] == [80, 144, 0, 0, 0]
    with pytest.raises(api.TvaError):
        api.kv4_record_bytes(32)


@pytest.mark.parametrize("fn", ["append_kv4", "read_kv4"])
def test_row_refusals(lib, fn):
    far = A + (1 << 30)

    def call(n=4, hkv=2, d=64, dtype=0, cap=16, k=far, v=far + (1 << 20), slot=A, cache=A, st=A):
        if fn == "append_kv4":
            return lib.append_kv4(n, hkv, d, dtype, cap, P(k), P(v), P(slot), P(cache), P(st), None)
        return lib.read_kv4(n, hkv, d, dtype, cap, P(cache), P(slot), P(k), P(v), P(st), None)
    assert call(n=0) == 0                                     # nothing to do, nothing launched
    assert call(n=-1) == 1 and call(hkv=0) == 1 and call(cap=-1) == 1 and call(cap=1 << 31) == 1
    assert call(d=96) == 2 and call(dtype=3) == 2
    assert call(k=None) == 1 and call(v=None) == 1 and call(cache=None) == 1 and call(st=None) == 1
    assert call(k=far + 8) == 1 and call(v=far + 4) == 1 and call(cache=A + 8) == 1
    assert call(k=A + 80) == 1 and call(v=A + 15 * 160) == 1  # inside the cache
    if fn == "append_kv4":
        assert call(slot=None) == 1
    else:
        assert call(v=far) == 1                               # k and v overlap


def test_commit_refusals(lib):
    row = 8 * 128 * 2

    def call(batch=1, hkv=8, d=128, dtype=0, ncap=16, maxn=16, cap=64, cu=A, ln=A, path=A, tk=A, tv=A + 16 * row, dst=A,
             cache=A + 64 * row, st=A):
        return lib.commit_accepted_kv4(batch, hkv, d, dtype, ncap, maxn, cap, P(cu), P(ln), P(path), P(tk), P(tv),
                                       P(dst), P(cache), P(st), None)
    assert call(batch=0) == 1 and call(hkv=0) == 1 and call(ncap=-1) == 1 and call(cap=-1) == 1
    assert call(d=96) == 2 and call(dtype=7) == 2
    assert call(maxn=0) == 1 and call(maxn=129) == 1
    for name in ("cu", "ln", "path", "tk", "tv", "dst", "cache", "st"):
        assert call(**{name: None}) == 1, name
    assert call(tk=A + 8) == 1 and call(cache=A + 8 * row) == 1


def test_the_binding_refuses_host_tensors_and_bad_types():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    rec = torch.zeros(4, 2, 80, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.append_kv4(x, x, i, rec)
    with pytest.raises(ValueError):
        api.read_kv4(rec, 64)
    with pytest.raises(ValueError):
        api.read_kv4(rec, 64, dtype=torch.float64)
    with pytest.raises(ValueError):
        api.commit_accepted_kv4(i, i, i, x, x, i, rec)
    with pytest.raises(ValueError):
        api.tree_verify_attn_kv4_varlen(x, rec, x, x, i, i, i, 4, 4)
    with pytest.raises(ValueError):
        api.tree_verify_attn_window_varlen(x, x, x, x, x, i, i, i, 4, 4, window=2)
