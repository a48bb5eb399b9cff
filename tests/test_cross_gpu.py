"""Cross-attention (cross_attn_varlen) against float64.  Bars: those of the tree attention
(tests/_gpu.py, TOL), whose arithmetic it shares: P rounded to 16 bits, one rounding of the output."""
import numpy as np
import pytest
import torch

import oracle
from tests._gpu import TOL
from tree_verification_attention_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()


class Problem:
    def __init__(self, dtype, keys, queries, heads, d, seed, spare=(0, 0)):
        self.dtype, self.keys, self.queries, (self.hq, self.hkv) = dtype, keys, queries, heads
        g = torch.Generator().manual_seed(seed)
        draw = lambda n, h, extra: torch.cat([torch.randn(n, h, d, generator=g), torch.full((extra, h, d), float("nan"))]).to(DT[dtype])  # noqa: E731,E501
        self.q, self.k, self.v = draw(sum(queries), self.hq, spare[1]), draw(sum(keys), self.hkv, spare[0]), draw(sum(keys), self.hkv, spare[0])  # noqa: E501
        cu = lambda a: torch.tensor(np.concatenate([[0], np.cumsum(a)]), dtype=torch.int32)  # noqa: E731
        self.cu_q, self.cu_k = cu(queries), cu(keys)
        self.dev = [x.cuda() for x in (self.q, self.k, self.v, self.cu_q, self.cu_k)]

    def run(self, status=0, **kw):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = api.cross_attn_varlen(*self.dev, max(self.queries), max(self.keys), dev_status=st, **kw)
        torch.cuda.synchronize()
        assert int(st.item()) == status
        return out, lse

    def check(self, out, lse):
        """Every row, with torch in float64 on the device (the oracle where it is small)."""
        n = sum(self.queries)
        ta, tl = TOL[self.dtype]
        q, k, v = (x.double() for x in self.dev[:3])
        for b, (m, P) in enumerate(zip(self.queries, self.keys)):
            i0, p0 = int(self.cu_q[b]), int(self.cu_k[b])
            o, l = out[i0:i0 + m].double(), lse[i0:i0 + m].double()
            if P == 0:
                assert (o == 0).all() and (l == -np.inf).all()
                continue
            G = self.hq // self.hkv
            z = torch.einsum("ihd,phd->ihp", q[i0:i0 + m], k[p0:p0 + P].repeat_interleave(G, 1)) / q.shape[2] ** 0.5
            l_ref = torch.logsumexp(z, -1)
            o_ref = torch.einsum("ihp,phd->ihd", (z - l_ref[..., None]).exp(), v[p0:p0 + P].repeat_interleave(G, 1))
            if m:
                assert (o - o_ref).abs().max() <= ta, float((o - o_ref).abs().max())
                assert ((l - l_ref).abs() / l_ref.abs().clamp(min=1)).max() <= tl
        assert n == 0 or torch.isfinite(out[:n].float()).all()


# (keys, queries, heads, d)
CASES = [
    ([1], [1], (4, 1), 64), ([0], [3], (4, 2), 64), ([128], [1], (32, 8), 128), ([129], [2], (32, 8), 128),
    ([127], [32], (8, 2), 64), ([1000], [16], (32, 8), 128), ([700], [200], (16, 2), 128),
    ([300], [333], (6, 2), 64), ([257], [1000], (8, 8), 128), ([0, 5, 0, 300, 128], [3, 1, 2, 0, 40], (12, 4), 64),
    ([513, 0, 1], [9, 300, 1], (8, 2), 128), ([40] * 20, [1] * 20, (32, 8), 128), ([0] * 17 + [9], [2] * 18, (4, 4), 64),
    ([640, 641, 5], [40, 40, 40], (32, 2), 128), ([0, 0], [5, 1], (4, 1), 128), ([90], [2500], (4, 1), 64),
    ([70, 71], [129, 500], (64, 2), 64), ([700], [400], (32, 8), 128), ([500], [2001], (8, 2), 128), ([260], [640], (8, 2), 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(dtype, case):
    keys, queries, heads, d = CASES[case]
    pr = Problem(dtype, keys, queries, heads, d, seed=case)
    pr.check(*pr.run())


def test_against_the_oracle():
    pr = Problem("fp32", [30, 0, 9], [2, 1, 3], (4, 2), 64, seed=3)
    out, lse = pr.run()
    o, l = oracle.cross_attention(*(x.double().numpy() for x in (pr.q, pr.k, pr.v)), pr.cu_q.numpy(), pr.cu_k.numpy(), 2)
    seen = np.isfinite(l)
    assert np.array_equal(seen, np.isfinite(lse.cpu().numpy()))
    assert np.abs(out.cpu().numpy() - o).max() <= 1e-4
    assert np.abs(lse.cpu().numpy()[seen] - l[seen]).max() <= 1e-5 * 5


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_random_shapes(dtype):
    rng = np.random.default_rng(8)
    for i in range(25):
        B = int(rng.integers(1, 24))
        keys = [int(x) for x in rng.integers(0, 700, B)]
        queries = [int(x) for x in 2 ** rng.uniform(0, 8 if dtype == "bf16" else 5, B)]
        heads = [(4, 1), (8, 8), (16, 2), (12, 4), (6, 2), (5, 5)][int(rng.integers(6))]
        pr = Problem(dtype, keys, queries, heads, int(rng.choice([64, 128])), seed=50 + i)
        pr.check(*pr.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_of_no_sequence(dtype):
    """NaN in cache rows and queries of no sequence is not seen, and output rows of none stay."""
    pr = Problem(dtype, [200, 0, 70], [5, 2, 33], (8, 2), 128, seed=4, spare=(300, 9))
    out = torch.full_like(pr.dev[0], 7.0)
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    pr.check(*pr.run(out=out, lse=lse))
    assert (out[40:] == 7.0).all() and (lse[40:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_neighbour_s_rows_do_not_leak(dtype):
    pr = Problem(dtype, [100, 60, 30], [4, 4, 4], (8, 2), 64, seed=5)
    for x in pr.dev[1:3]:
        x[100:160] = float("inf")
    out, lse = pr.run()
    keep = Problem(dtype, [100, 30], [4, 4], (8, 2), 64, seed=5)
    pick = torch.tensor([*range(4), *range(8, 12)], device="cuda")
    keep.dev = [pr.dev[0][pick].contiguous(), *(x[[*range(100), *range(160, 190)]].contiguous() for x in pr.dev[1:3]), *keep.dev[3:]]
    keep.check(out[pick], lse[pick])


def test_scale_bounds_plan_and_a_small_workspace():
    pr = Problem("bf16", [300, 40], [6, 3], (8, 2), 128, seed=6)
    q, k, v, cu_q, cu_k = pr.dev
    out, lse = api.cross_attn_varlen(q, k, v, cu_q, cu_k, 6, 300, softmax_scale=0.02)
    z = torch.einsum("ihd,phd->ihp", q[:6].double(), k[:300].double().repeat_interleave(4, 1)) * 0.02
    torch.cuda.synchronize()
    assert (lse[:6].double() - torch.logsumexp(z, -1)).abs().max() <= 1e-3 * 7
    p = api.make_params(q, k, cu_k, cu_q, 2, 300, 6)
    ws = api.alloc_cross_workspace(p, q.device)
    a, b = pr.run(params=p, workspace=ws), pr.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(api.TvaError):
        pr.run(workspace=ws[: ws.numel() - 256])
    with pytest.raises(ValueError):
        pr.run(params=p, softmax_scale=0.5)
    with pytest.raises(ValueError):
        api.cross_attn_varlen(q[:8], k, v, cu_q, cu_k, 6, 300, params=p)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bounds_are_reported_and_the_other_sequences_run(dtype):
    """A sequence with more keys or queries than stated is skipped; its rows are unspecified."""
    pr = Problem(dtype, [50, 200, 30], [3, 4, 9], (8, 2), 64, seed=7)
    q, k, v, cu_q, cu_k = pr.dev
    for queries, keys in ((9, 199), (8, 200)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = api.cross_attn_varlen(q, k, v, cu_q, cu_k, queries, keys, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 1
        only = Problem(dtype, [50], [3], (8, 2), 64, seed=7)
        only.dev = [q[:3].contiguous(), k[:50].contiguous(), v[:50].contiguous(), *only.dev[3:]]
        only.check(out[:3], lse[:3])


def test_captured_replayed_and_on_two_streams():
    prs = [Problem("bf16", [700, 3], [20, 5], (16, 2), 128, seed=8), Problem("fp16", [300], [150], (8, 2), 64, seed=9)]
    alone = [p.run() for p in prs]
    for p, (o_ref, l_ref) in zip(prs, alone):
        plan = api.make_params(p.dev[0], p.dev[1], p.dev[4], p.dev[3], p.hkv, max(p.keys), max(p.queries))
        ws = api.alloc_cross_workspace(plan, p.dev[0].device)
        out, lse, st = torch.empty_like(o_ref), torch.empty_like(l_ref), torch.zeros(1, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.cross_attn_varlen(*p.dev, max(p.queries), max(p.keys), out=out, lse=lse, workspace=ws, dev_status=st)
        for _ in range(3):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o_ref) and torch.equal(lse, l_ref)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [api.cross_attn_varlen(*p.dev, max(p.queries), max(p.keys), stream=s) for p, s in zip(prs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_it_is_the_tree_attention_s_prefix_part():
    """Merged with the tree keys' own part by the log-sum-exp rule it gives the hybrid attention."""
    pr = Problem("fp32", [400], [6], (8, 2), 128, seed=10)
    q, k, v, cu_q, cu_k = pr.dev
    g = torch.Generator().manual_seed(11)
    tk, tv = (torch.randn(6, 2, 128, generator=g).cuda() for _ in range(2))
    parent = torch.tensor([-1, 0, 0, 1, 1, 2], dtype=torch.int32, device="cuda")
    whole, l = api.tree_verify_attn_varlen(q, k, v, tk, tv, parent, cu_k, cu_q, 400, 6)
    o1, l1 = pr.run()
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    o2, l2 = api.tree_verify_attn_varlen(q, k, v, tk, tv, parent, none, cu_q, 0, 6)
    both = torch.logaddexp(l1, l2)
    got = o1 * (l1 - both).exp()[..., None] + o2 * (l2 - both).exp()[..., None]
    assert (got - whole).abs().max() <= 2e-4 and (both - l).abs().max() <= 1e-4
