"""A kept plan (``params=``) of the windowed and 4-bit-cache forms: what does not belong to the
call is refused before anything is launched, and a plan's scale is the one that is used."""
import numpy as np
import pytest
import torch

from tests import _window
from tree_verification_attention_gb300 import api


def _tensors(device, B=3, spare=0):
    """A batch of B sequences (4 rows, 2 nodes each) in arrays that may be longer."""
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
    cu = lambda n: torch.arange(0, n * (B + spare + 1), n, dtype=torch.int32, device=device)  # noqa: E731
    N = 2 * B
    return dict(q=z(N, 8, 64), cache=z(4 * B, 2, 64), tree=z(N, 2, 64), cu_prefix=cu(4), cu_nodes=cu(2),
                parent=torch.tensor([-1, 0] * B, dtype=torch.int32, device=device))


def _plan(t, B, **kw):
    a = dict(max_prefix_len=4, max_nodes=2, softmax_scale=0.0)
    a.update(kw)
    return api.make_params(t["q"], t["cache"], t["cu_prefix"][:B + 1], t["cu_nodes"][:B + 1], 2, **a)


def _check(t, p, B, max_prefix_len=4, max_nodes=2, softmax_scale=0.0, reported=False):
    api._check_plan(p, t["q"], 2, t["cache"].shape[0], t["cu_prefix"][:B + 1], t["cu_nodes"][:B + 1], max_prefix_len,
                    max_nodes, softmax_scale, reported)


def test_a_plan_of_the_same_call_is_taken():
    t = _tensors("cpu")
    _check(t, _plan(t, 3), 3)
    _check(t, _plan(t, 3, max_prefix_len=9, max_nodes=7), 3)      # bounds may be generous
    _check(t, _plan(t, 3), 3, None, None)                         # none named: the plan's
    for s in (0.3, 1.0 / 3.0, 7.0):
        _check(t, _plan(t, 3, softmax_scale=s), 3, softmax_scale=s)
        _check(t, _plan(t, 3, softmax_scale=s), 3)                # no scale given: the plan's
    _check(t, _plan(t, 3), 3, softmax_scale=64 ** -0.5)           # the default, spelled out


@pytest.mark.parametrize("mine,plans", [(2, 3), (3, 2), (1, 3), (3, 4)])
def test_a_plan_of_another_batch_is_refused(mine, plans):
    """Slices of one array share its address."""
    t = _tensors("cpu", spare=1)
    p = _plan(t, plans)
    assert p.cu_prefix == t["cu_prefix"][:mine + 1].data_ptr() and p.cu_nodes == t["cu_nodes"][:mine + 1].data_ptr()
    with pytest.raises(ValueError, match="do not describe"):
        _check(t, p, mine, reported=True)


@pytest.mark.parametrize("given,plans", [(0.5, 0.0), (0.125, 0.25), (0.0884, 0.0883), (1.0, 0.125)])
def test_another_scale_is_refused(given, plans):
    t = _tensors("cpu")
    with pytest.raises(ValueError, match="softmax_scale"):
        _check(t, _plan(t, 3, softmax_scale=plans), 3, softmax_scale=given, reported=True)


def test_lengths_beyond_the_plan_are_refused_where_no_status_word_tells():
    t = _tensors("cpu")
    for p in (_plan(t, 3, max_prefix_len=3), _plan(t, 3, max_nodes=1)):
        with pytest.raises(ValueError, match="shorter prefixes or smaller trees"):
            _check(t, p, 3)
        _check(t, p, 3, reported=True)  # the device reports the sequence that does not fit


@pytest.mark.parametrize("change", [dict(num_q_heads=4), dict(num_kv_heads=4), dict(head_dim=128), dict(dtype=2),
                                    dict(node_capacity=7), dict(kv_capacity=13), dict(cu_prefix=64),
                                    dict(cu_nodes=64)])
def test_a_plan_of_other_tensors_is_refused(change):
    t = _tensors("cpu")
    p = _plan(t, 3)
    for k, v in change.items():
        setattr(p, k, v)
    with pytest.raises(ValueError, match="do not describe"):
        _check(t, p, 3, reported=True)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.gpu
@pytest.mark.parametrize("kv4", [False, True])
def test_the_calls_refuse_what_the_check_refuses(lib, kv4):
    pr = _window.Problem("bf16", [40, 9, 20], [5, 3, 4], (8, 2), 64, "random", seed=60, kv4=kv4)
    t = pr.device()
    cache = t["kv4_cache"] if kv4 else t["k_cache"]
    part = dict(t, cu_prefix=t["cu_prefix"][:3], cu_nodes=t["cu_nodes"][:3])
    whole = api.make_params(t["q"], cache, t["cu_prefix"], t["cu_nodes"], 2, pr.max_prefix, pr.max_nodes)
    two = api.make_params(t["q"], cache, part["cu_prefix"], part["cu_nodes"], 2, pr.max_prefix, pr.max_nodes)
    for tensors, plan in ((part, whole), (t, two)):
        with pytest.raises(ValueError, match="do not describe"):
            pr.call(tensors, 16, 1, params=plan)
    with pytest.raises(ValueError, match="softmax_scale"):
        pr.call(t, 16, 1, params=whole, softmax_scale=0.5)
    for short in (dict(max_prefix_len=39, max_nodes=5), dict(max_prefix_len=40, max_nodes=4)):
        plan = api.make_params(t["q"], cache, t["cu_prefix"], t["cu_nodes"], 2, **short)
        with pytest.raises(ValueError, match="shorter prefixes or smaller trees"):
            pr.call(t, 16, 1, params=plan)
    out, lse = pr.call(t, 16, 1, params=whole)
    pr.check(out, lse, 16, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("dtype,kv4,window", [("bf16", False, 60), ("fp32", False, 60), ("fp16", True, 0),
                                              ("bf16", True, 60)])
@pytest.mark.parametrize("scale", [0.05, 0.5])
def test_a_scale_of_the_callers(lib, dtype, kv4, window, planned, scale):
    """The default scale over q times scale sqrt(d) is the same attention; with d = 64 and
    these scales the factor (0.4, 4) is taken in float64, on the reference's side."""
    pr = _window.Problem(dtype, [150, 0, 33], [6, 20, 1], (8, 2), 64, "random", seed=61, kv4=kv4)
    t = pr.device()
    cache = t["kv4_cache"] if kv4 else t["k_cache"]
    more = dict(softmax_scale=scale)
    if planned:
        more = dict(params=api.make_params(t["q"], cache, t["cu_prefix"], t["cu_nodes"], 2, pr.max_prefix, pr.max_nodes,
                                           softmax_scale=scale))
    out, lse = pr.call(t, window, 2, **more)
    torch.cuda.synchronize()
    # the scale reaches the kernel as a float32; its rounding is within the tolerance's logit error
    factor = float(np.float32(scale)) * 8.0
    pr.q = pr.q.double() * factor
    pr.check(out, lse, window, 2)
