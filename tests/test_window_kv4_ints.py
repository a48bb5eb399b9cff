"""Whole-number arguments of the windowed and 4-bit-cache calls: a C int holds 32 bits, and a
value that does not fit is refused instead of arriving as its low bits."""
import pytest
import torch

import __graft_entry__
from tree_verification_attention_gb300 import api

TOO_WIDE = [2 ** 31, 2 ** 32, 2 ** 32 + 8, -2 ** 31 - 1, 2 ** 70]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def _calls(**kw):
    """Both attention forms with one argument changed (host tensors: a call that takes the
    number ends at the next check, which names the tensor)."""
    x, rec = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 80, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    a = dict(max_prefix_len=4, max_nodes=4, window=2, sinks=1)
    a.update(kw)
    yield lambda: api.tree_verify_attn_window_varlen(x, x, x, x, x, i, i, i, **a)
    yield lambda: api.tree_verify_attn_kv4_varlen(x, rec, x, x, i, i, i, **a)


@pytest.mark.parametrize("name", ["window", "sinks", "max_prefix_len", "max_nodes"])
@pytest.mark.parametrize("value", TOO_WIDE + [2.5])
def test_attention(name, value):
    for call in _calls(**{name: value}):
        with pytest.raises(ValueError, match=f"{name} = .*32-bit whole number"):
            call()


@pytest.mark.parametrize("name", ["window", "sinks", "max_prefix_len", "max_nodes"])
@pytest.mark.parametrize("value", [2 ** 31 - 1, 7, 7.0])
def test_attention_takes_what_fits(name, value):
    for call in _calls(**{name: value}):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("value", TOO_WIDE)
def test_commit(value):
    x, rec = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 80, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_nodes = .*32-bit whole number"):
        api.commit_accepted_kv4(i, i, i, x, x, i, rec, max_nodes=value)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.commit_accepted_kv4(i, i, i, x, x, i, rec, max_nodes=4)


@pytest.mark.parametrize("d", [64, 128])
def test_head_dim(d):
    for value in (d + 2 ** 32, d - 2 ** 32, d + 0.5):
        with pytest.raises(ValueError, match="head_dim = .*32-bit whole number"):
            api.kv4_record_bytes(value)
    assert api.kv4_record_bytes(d) == (80 if d == 64 else 144)
