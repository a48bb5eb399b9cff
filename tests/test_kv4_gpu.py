"""The 4-bit cache on the GPU: writing, reading, committing, and the attention over it."""
import numpy as np
import pytest
import torch

import oracle
from tests import _window
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu

DTYPES = _window.DTYPES


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _rows(kind, dt, n, hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(n, hkv, d, generator=g) for _ in range(2))
    if kind == "wide":      # magnitudes over many binades, blocks of zeros and of tiny values
        k *= 2.0 ** torch.randint(-22, 15, (n, hkv, 1), generator=g)
        v *= 2.0 ** torch.randint(-22, 15, (n, hkv, 1), generator=g)
        v[:, :, :16] = 0
    elif kind == "ties":    # halves of a scale, and scales halfway between two
        k = torch.randint(-15, 16, (n, hkv, d), generator=g) * 0.5 * torch.randint(8, 16, (n, hkv, 1), generator=g)
        v = torch.randint(-15, 16, (n, hkv, d), generator=g) * 0.5 * 2.0 ** -17
        k[:, :, ::16] = 7 * (torch.randint(8, 16, (n, hkv, d // 16), generator=g) + 0.5)
    elif kind == "next to ties" and dt == torch.float32:
        k = torch.randint(-15, 16, (n, hkv, d), generator=g) * 0.5 * torch.randint(8, 16, (n, hkv, 1), generator=g)
        k = torch.nextafter(k.float(), torch.where(torch.rand(n, hkv, d, generator=g) < 0.5, -1e9, 1e9))
        v = 7 * (torch.randint(8, 16, (n, hkv, d), generator=g) + 0.5)
        v = torch.nextafter(v.float(), torch.where(torch.rand(n, hkv, d, generator=g) < 0.5, -1e9, 1e9))
    elif kind == "special":
        k[0, 0, 3], k[0, 0, 20], k[1, 0, 40] = float("nan"), float("inf"), -float("inf")
        v[:2], v[2, :, 5] = float("nan"), 60000.0
    return k.to(dt), v.to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["plain", "wide", "ties", "next to ties", "special"])
def test_append_writes_the_records_bit_for_bit(dtype, d, kind):
    n, hkv, cap = 37, 3, 60
    k, v = _rows(kind, DTYPES[dtype], n, hkv, d)
    rng = np.random.default_rng(1)
    slot = rng.permutation(cap)[:n].astype(np.int32)
    slot[[4, 30]] = -1
    before = torch.randint(0, 256, (cap, hkv, api.kv4_record_bytes(d)), dtype=torch.uint8,
                           generator=torch.Generator().manual_seed(2))
    cache = before.cuda()
    st = api.append_kv4(k.cuda(), v.cuda(), _i32(slot), cache)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want = before.numpy().copy()
    rec = oracle.kv4_pack(k.double().numpy(), v.double().numpy())
    for i, s in enumerate(slot):
        if s >= 0:
            want[s] = rec[i]
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_every_bf16_and_fp16_value_beside_every_scale():
    """Each finite 16-bit value once in a block whose largest magnitude is drawn."""
    for dt in (torch.bfloat16, torch.float16):
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
        x = x[torch.isfinite(x.float())]
        x = x[torch.argsort(x.float().abs(), stable=True)]
        x = torch.nn.functional.pad(x, (0, -x.numel() % 1024)).view(-1, 1, 64)
        k = torch.flip(x, (2,)).contiguous()
        slot = torch.arange(x.shape[0], dtype=torch.int32, device="cuda")
        cache = api.alloc_kv4_cache(x.shape[0], 1, 64)
        api.append_kv4(k.cuda(), x.cuda(), slot, cache)
        assert np.array_equal(cache.cpu().numpy(), oracle.kv4_pack(k.double().numpy(), x.double().numpy()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (2, 128), (8, 128)])
def test_read_gives_the_values_exactly(dtype, hkv, d):
    k, v = _rows("wide", torch.float32, 45, hkv, d, seed=3)
    rec = oracle.kv4_pack(k.double().numpy(), v.double().numpy())
    K, V = oracle.kv4_values(rec, d)
    cache = torch.from_numpy(rec).cuda()
    gk, gv = api.read_kv4(cache, d, dtype=DTYPES[dtype])
    assert np.array_equal(gk.double().cpu().numpy(), K) and np.array_equal(gv.double().cpu().numpy(), V)
    slot = [44, 0, -1, 7, 7, 45, 3]   # padding reads as zeros, rows may repeat, 45 is outside
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gk, gv = api.read_kv4(cache, d, slot=_i32(slot), dtype=DTYPES[dtype], dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 1
    for got, ref in ((gk, K), (gv, V)):
        want = np.stack([ref[s] if 0 <= s < 45 else np.zeros_like(ref[0]) for s in slot])
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_append_reports_rows_outside_and_writes_the_others():
    k, v = _rows("plain", torch.bfloat16, 3, 2, 64)
    cache = api.alloc_kv4_cache(5, 2, 64)
    st = api.append_kv4(k.cuda(), v.cuda(), _i32([1, 5, 2 ** 31 - 1]), cache)
    torch.cuda.synchronize()
    assert int(st.item()) == 1
    want = np.zeros((5, 2, 80), np.uint8)
    want[1] = oracle.kv4_pack(k.double().numpy(), v.double().numpy())[0]
    assert np.array_equal(cache.cpu().numpy(), want)
    none = api.append_kv4(k[:0].cuda(), v[:0].cuda(), _i32([]), cache)  # no rows: nothing to do
    assert int(none.item()) == 0 and api.read_kv4(cache, 64, slot=_i32([]))[0].shape == (0, 2, 64)


def test_append_past_32_bits_of_bytes():
    """A cache of more than 2^32 bytes: records at its far end."""
    rows, hkv, d = 3_900_000, 8, 128
    cache = torch.empty((rows, hkv, 144), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    k, v = _rows("plain", torch.bfloat16, 4, hkv, d, seed=4)
    slot = [0, rows - 1, rows - 129, 2 ** 32 // (8 * 144) + 1]
    st = api.append_kv4(k.cuda(), v.cuda(), _i32(slot), cache)
    gk, gv = api.read_kv4(cache, d, slot=_i32(slot), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    K, V = oracle.kv4_values(oracle.kv4_pack(k.double().numpy(), v.double().numpy()), d)
    assert np.array_equal(gk.double().cpu().numpy(), K) and np.array_equal(gv.double().cpu().numpy(), V)


def test_attention_past_32_bits_of_bytes():
    """A sequence at the far end of a cache of more than 2^32 bytes."""
    rows, at, P = 3_900_000, 3_899_000, 700
    pr = _window.Problem("bf16", [P], [9], (32, 8), 128, "random", seed=5, kv4=True)
    cache = torch.empty((rows, 8, 144), dtype=torch.uint8, device="cuda")
    cache[at:at + P] = pr.records[:P].cuda()
    t = pr.device()
    for window, sinks in ((0, 0), (300, 4)):
        # sequence 0 is long and has no nodes: its rows are not read
        out, lse = api.tree_verify_attn_kv4_varlen(t["q"], cache, t["tree_k"], t["tree_v"], t["parent"],
                                                   _i32([0, at, at + P]), _i32([0, 0, 9]), at, 9, window=window,
                                                   sinks=sinks)
        torch.cuda.synchronize()
        pr.check(out, lse, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("hkv,d", [(3, 64), (8, 128)])
def test_commit_quantises_the_accepted_rows(dtype, hkv, d):
    rng = np.random.default_rng(7)
    sizes = [32, 0, 1, 128, 7]
    N, B = sum(sizes), len(sizes)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    k, v = _rows("plain", DTYPES[dtype], N, hkv, d, seed=6)
    lens = np.array([5, 0, 1, 40, 7], np.int32)
    path = np.full(N, -1, np.int32)
    for b in range(B):
        path[cu[b]:cu[b] + lens[b]] = np.sort(rng.permutation(sizes[b])[:lens[b]])
    dst = np.array([3, 0, 160, 20, 90], np.int32)
    before = torch.randint(0, 256, (161, hkv, api.kv4_record_bytes(d)), dtype=torch.uint8)
    cache = before.cuda()
    args = (_i32(cu), _i32(lens), _i32(path), k.cuda(), v.cuda(), _i32(dst))
    st = api.commit_accepted_kv4(*args, cache)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    rec = oracle.kv4_pack(k.double().numpy(), v.double().numpy())
    want, _ = oracle.commit_accepted_kv(before.numpy(), before.numpy(), rec, rec, cu, lens, path, dst)
    assert np.array_equal(cache.cpu().numpy(), want)
    # a sequence out of bounds is left alone, the others are written
    for name, value in (("dst", 161), ("lens", 33), ("lens", -1), ("path", 32)):
        a = dict(lens=lens.copy(), path=path.copy(), dst=dst.copy())
        a[name][0] = value
        cache = before.cuda()
        st = api.commit_accepted_kv4(_i32(cu), _i32(a["lens"]), _i32(a["path"]), args[3], args[4], _i32(a["dst"]), cache)
        torch.cuda.synchronize()
        got = cache.cpu().numpy()
        assert int(st.item()) == 1
        assert np.array_equal(got[3:8], before.numpy()[3:8]) and np.array_equal(got[20:60], want[20:60])


# (prefixes, nodes, heads, d, tree, window, sinks)
CASES = [
    ([0], [1], (4, 1), 64, "chain", 0, 0),
    ([1], [1], (4, 4), 128, "chain", 0, 0),
    ([1000], [1], (32, 8), 128, "chain", 0, 0),                  # a single token
    ([129], [8], (32, 8), 128, "chain", 0, 0),
    ([3000], [64], (32, 8), 128, "random", 0, 0),
    ([2000], [68], (32, 8), 128, "random", 0, 0),                # several row groups, teams of workers
    ([900], [128], (64, 8), 128, "random", 0, 0),
    ([513, 0, 127, 128, 129, 1], [9, 3, 1, 17, 2, 5], (8, 2), 64, "random", 0, 0),
    ([300, 40, 260], [5, 0, 33], (12, 4), 128, "random", 0, 0),   # an empty tree; G = 3
    ([640, 641, 5], [40, 40, 40], (32, 2), 128, "random", 0, 0),  # G = 16
    ([600, 90], [100, 128], (4, 4), 64, "chain", 0, 0),
    ([300], [8], (8, 2), 64, "chain", 100, 4),
    ([700], [128], (16, 2), 128, "chain", 5, 0),
    ([700], [128], (16, 2), 128, "chain", 5, 130),
    ([513, 0, 127, 128, 129, 1], [9, 3, 1, 17, 2, 5], (8, 2), 64, "random", 127, 128),
    ([640, 641, 5], [40, 40, 40], (32, 2), 128, "random", 260, 129),
    ([1500], [33], (32, 8), 128, "random", 2 ** 31 - 1, 4),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_against_the_definition(dtype, case):
    P, m, heads, d, kind, window, sinks = CASES[case]
    pr = _window.Problem(dtype, P, m, heads, d, kind, seed=200 + case, kv4=True)
    out, lse = pr.run(window, sinks)
    pr.check(out, lse, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_over_many_random_shapes(dtype):
    rng = np.random.default_rng(9)
    for i in range(30):
        B = int(rng.integers(1, 12))
        P = [int(x) for x in rng.integers(0, 900, B)]
        m = [int(x) for x in rng.integers(0, 40, B)]
        m[0] = max(1, m[0])
        heads = [(4, 1), (8, 8), (16, 2), (12, 4), (6, 2)][int(rng.integers(5))]
        window, sinks = int(rng.choice([0, int(2 ** rng.uniform(0, 10))])), int(rng.choice([0, 1, 4, 64, 131]))
        pr = _window.Problem(dtype, P, m, heads, int(rng.choice([64, 128])), str(rng.choice(["chain", "random"])),
                             seed=i, kv4=True)
        out, lse = pr.run(window, sinks)
        pr.check(out, lse, window, sinks, (i, P, m, heads, window, sinks))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_code_and_every_scale_reaches_the_attention(dtype):
    """Values through V: with zero queries every visible key has the same weight, so a
    one-key prefix of value x and a tree value of 0 give x / 2 (or x rounded once)."""
    d, n = 64, 211
    codes = np.arange(16, dtype=np.uint32)
    rec = np.zeros((n, 1, 80), np.uint8)
    word = sum((codes[e:e + 9:8].astype(np.uint32)) << np.uint32(4 * (e // 2) + 16 * (e % 2)) for e in range(8))
    rec[:, 0, 32:64] = np.tile(word.astype("<u4").view(np.uint8), 4)      # V: codes 0 .. 15 in each block
    rec[:, 0, 68:72] = np.arange(n, dtype=np.uint8)[:, None]              # V scales
    K, V = oracle.kv4_values(rec, d)
    dt = DTYPES[dtype]
    z = torch.zeros(n, 1, d, dtype=dt, device="cuda")
    ar = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse = api.tree_verify_attn_kv4_varlen(z, torch.from_numpy(rec).cuda(), z, z,
                                               torch.full((n,), -1, dtype=torch.int32, device="cuda"), ar, ar, 1, 1)
    torch.cuda.synchronize()
    half = torch.from_numpy(V / 2).to(dt).double().numpy()
    assert np.array_equal(out.double().cpu().numpy(), half)
    assert np.abs(lse.cpu().numpy() - np.log(2)).max() < 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nodes", [[3, 20], [40, 100]])
def test_records_that_no_node_sees_may_hold_anything(dtype, nodes):
    pr = _window.Problem(dtype, [400, 333], nodes, (8, 2), 128, "random", seed=3, spare=200, kv4=True)
    for window, sinks in ((0, 0), (70, 5)):
        rec = pr.records.clone()
        if window:
            for p0, P in ((0, 400), (400, 333)):
                rec[p0 + sinks:p0 + P - window + 1] = 255
        rec[733:] = 255
        t = dict(pr.device(), kv4_cache=rec.cuda())
        out, lse = pr.run(window, sinks, t)
        pr.check(out, lse, window, sinks)


def test_nan_tree_rows_of_another_sequence_do_not_spread():
    pr = _window.Problem("bf16", [200, 300], [5, 6], (8, 2), 128, "chain", seed=13, kv4=True)
    t = pr.device()
    t["tree_v"][5:] = float("nan")
    out, lse = pr.call(t, 0, 0)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[:5].float()).all()) and bool(torch.isnan(out[5:].float()).all())


def test_a_verification_cycle_over_the_4_bit_cache():
    """Prefill rows appended; the tree's attention; the walk; the commit; and the next
    step's attention over what the cache then holds, all against float64."""
    B, hkv, hq, d, m, room = 3, 2, 8, 128, 12, 40
    rng = np.random.default_rng(14)
    prefix = [150, 3, 270]
    start = np.concatenate([[0], np.cumsum([p + room for p in prefix])])
    cache = api.alloc_kv4_cache(int(start[-1]), hkv, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(15)
    draw = lambda n, h: torch.randn(n, h, d, generator=g).to(torch.bfloat16)  # noqa: E731
    held = [None] * B
    for b, P in enumerate(prefix):
        k, v = draw(P, hkv), draw(P, hkv)
        api.append_kv4(k.cuda(), v.cuda(), torch.arange(start[b], start[b] + P, dtype=torch.int32, device="cuda"), cache,
                       dev_status=st)
        held[b] = oracle.kv4_values(oracle.kv4_pack(k.double().numpy(), v.double().numpy()), d)
    for step in range(3):
        window, sinks = ((0, 0), (64, 4), (0, 0))[step]
        parent = np.concatenate([_window.tree(rng, "random", m) for _ in range(B)])
        q, tk, tv = draw(B * m, hq), draw(B * m, hkv), draw(B * m, hkv)
        cu_nodes = np.arange(0, B * m + 1, m, dtype=np.int32)
        # the cache's sequences have room between them: each is a problem of its own
        for b in range(B):
            sl = slice(b * m, (b + 1) * m)
            at = int(start[b])
            out, lse = api.tree_verify_attn_kv4_varlen(
                q[sl].cuda(), cache[at:at + prefix[b] + room], tk[sl].cuda(), tv[sl].cuda(), _i32(parent[sl]),
                _i32([0, prefix[b]]), _i32([0, m]), prefix[b], m, window=window, sinks=sinks, dev_status=st)
            ref, L, w = oracle.tree_verify_window_attention(
                q[sl].double().numpy(), *held[b], [0, prefix[b]], tk[sl].double().numpy(), tv[sl].double().numpy(),
                parent[sl], [0, m], hkv, window, sinks)
            # one rounding of the weights, one of the output, each at most 2^-8; fp32 sums far below
            assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -8 * (1.01 * w + np.abs(ref)) + 1e-6).all()
            assert np.abs(lse.double().cpu().numpy() - L).max() < 1e-4
        draft = rng.integers(0, 3, B * m).astype(np.int32)
        target = rng.integers(0, 3, B * m + B).astype(np.int32)
        alen, apath, _ = api.accept_longest_path(_i32(cu_nodes), _i32(parent), _i32(draft), _i32(target), dev_status=st)
        dst = [int(start[b]) + prefix[b] for b in range(B)]
        api.commit_accepted_kv4(_i32(cu_nodes), alen, apath, tk.cuda(), tv.cuda(), _i32(dst), cache, max_nodes=m,
                                dev_status=st)
        torch.cuda.synchronize()
        lens, paths = alen.tolist(), apath.tolist()
        for b in range(B):
            rows = [b * m + paths[b * m + j] for j in range(lens[b])]
            if rows:
                new = oracle.kv4_values(oracle.kv4_pack(tk[rows].double().numpy(), tv[rows].double().numpy()), d)
                held[b] = tuple(np.concatenate([x, y]) for x, y in zip(held[b], new))
            prefix[b] += lens[b]
            gk, gv = api.read_kv4(cache, d, slot=torch.arange(start[b], start[b] + prefix[b], dtype=torch.int32,
                                                              device="cuda"))
            assert np.array_equal(gk.double().cpu().numpy(), held[b][0])
            assert np.array_equal(gv.double().cpu().numpy(), held[b][1])
    assert int(st.item()) == 0


def test_a_captured_cycle_replays():
    """append, attention and commit captured into one graph; replayed on new inputs."""
    pr, other = (_window.Problem("fp16", [300, 90], [10, 4], (16, 2), 64, "chain", seed=s, kv4=True) for s in (16, 17))
    t, new = pr.device(), other.device()
    R = pr.records.shape[0]
    k, v = pr.k[:390].cuda(), pr.v[:390].cuda()
    slot = torch.arange(390, dtype=torch.int32, device="cuda")
    cache = api.alloc_kv4_cache(R + 20, 2, 64)
    p = api.make_params(t["q"], cache, t["cu_prefix"], t["cu_nodes"], 2, 300, 10)
    ws = api.alloc_workspace(p, "cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device="cuda")
    alen, apath, dst = _i32([2, 1]), _i32([0, 1] + [-1] * 8 + [0, -1, -1, -1]), _i32([R, R + 10])

    def cycle():
        api.append_kv4(k, v, slot, cache, dev_status=st)
        api.tree_verify_attn_kv4_varlen(t["q"], cache, t["tree_k"], t["tree_v"], t["parent"], t["cu_prefix"],
                                        t["cu_nodes"], 300, 10, window=200, sinks=4, out=out, lse=lse, workspace=ws,
                                        dev_status=st, params=p)
        api.commit_accepted_kv4(t["cu_nodes"], alen, apath, t["tree_k"], t["tree_v"], dst, cache, max_nodes=10,
                                dev_status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cycle()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        cycle()
    for name in ("q", "tree_k", "tree_v", "parent"):
        t[name].copy_(new[name])
    k.copy_(other.k[:390])
    v.copy_(other.v[:390])
    cache.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    other.check(out, lse, 200, 4)
    rec = oracle.kv4_pack(other.tree_k.double().numpy(), other.tree_v.double().numpy())
    got = cache.cpu().numpy()
    assert np.array_equal(got[R:R + 2], rec[:2]) and np.array_equal(got[R + 10], rec[10])
    assert np.array_equal(got[:390], other.records[:390].numpy())


def test_the_binding_refuses_what_does_not_fit():
    pr = _window.Problem("bf16", [100], [4], (8, 2), 64, "chain", seed=18, kv4=True)
    t = pr.device()
    with pytest.raises(api.TvaError) as e:
        pr.call(dict(t, q=t["q"].float(), tree_k=t["tree_k"].float(), tree_v=t["tree_v"].float()), 0, 0)
    assert e.value.code == 2
    with pytest.raises(api.TvaError):
        pr.call(t, -1, 0)
    for cache in (t["kv4_cache"][:, :, :72].contiguous(), t["kv4_cache"].view(torch.int8), t["kv4_cache"][:, :1],
                  t["kv4_cache"].cpu()):
        with pytest.raises(ValueError):
            pr.call(dict(t, kv4_cache=cache), 0, 0)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        api.append_kv4(k, k.half(), _i32([0, 1, 2, 3]), t["kv4_cache"])
    with pytest.raises(ValueError):
        api.append_kv4(k, k, _i32([0, 1, 2]), t["kv4_cache"])
    with pytest.raises(ValueError):
        api.append_kv4(k, k, _i32([0, 1, 2, 3]).long(), t["kv4_cache"])
    with pytest.raises(ValueError):
        api.append_kv4(k.transpose(0, 1), k.transpose(0, 1), _i32([0, 1]), t["kv4_cache"])
    with pytest.raises(ValueError):
        api.read_kv4(t["kv4_cache"], 128)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("seed", range(6))
def test_batches_of_short_sequences_agree_call_after_call(dtype, seed):
    """Workers whose ranges cross several short row groups, in batches large enough for the
    staged running sums: right, and the same bits every time."""
    rng = np.random.default_rng(60 + seed)
    B = int(rng.integers(16, 48))
    P = [int(x) for x in rng.integers(0, (100, 300, 2000)[seed % 3], B)]
    m = [int(x) for x in rng.integers(0, 9 if seed % 2 else 50, B)]
    m[0] = 1
    heads, d = [((12, 4), 128), ((8, 2), 64), ((32, 8), 128)][seed % 3]
    pr = _window.Problem(dtype, P, m, heads, d, "random", seed=seed, kv4=True)
    t = pr.device()
    for window, sinks in ((0, 0), (60, 4)):
        out, lse = pr.run(window, sinks, t)
        pr.check(out, lse, window, sinks, (B, P, m))
        for _ in range(10):
            again = pr.run(window, sinks, t)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
