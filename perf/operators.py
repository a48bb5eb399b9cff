"""The measured cases of the windowed and 4-bit-cache operators of tree verification.

Four operators, reached through ``tree_verification_attention_gb300.api``:

* ``tree_verify_attn_window_varlen``: tree-verification attention in which a node at
  position t sees the key at position s when t - s < window or s < sinks;
* ``tree_verify_attn_kv4_varlen``: tree-verification attention over a prefix cache held
  in 4 bits (whole prefix, or with a window and sinks);
* ``append_kv4`` / ``read_kv4``: K / V rows quantised into the 4-bit cache, and the
  values that its records stand for;
* ``commit_accepted_kv4``: the accepted path's K / V rows quantised into the cache.

The 4-bit cache is [rows, Hkv, record] bytes; a record holds one row's K and V of one
head: d / 2 bytes of K codes, d / 2 of V codes, d / 16 K scales, d / 16 V scales, padded
to a multiple of 16.  The little-endian 32-bit code word i holds elements 8 i .. 8 i + 7:
element 8 i + 2 j in bits 4 j .. 4 j + 3, element 8 i + 2 j + 1 in bits 16 + 4 j .. A code
n stands for (n - 8) times its block's scale (16 elements a block); a scale byte is an
unsigned float of 5 exponent bits (bias 15, with subnormals) and 3 mantissa bits, at
most 2560.  A block's scale is its largest magnitude over 7, rounded to nearest (ties to
even); a code is the value over the scale, rounded to nearest (ties to even), limited to
-7 .. 7.

Each case is a plain dict; the comments in ``listed`` say what it stands for.
"""
import math
import random

import torch

own = False  # True: run() calls the framework's operators; False: their plain form

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCALE_MAX = 2560.0


# ------------------------------------------------------------------------- the cases

def listed():
    attn = dict(op="kv4", dtype="bf16", batch=1, prefix_lo=16384, prefix_hi=16384, nodes=8, tree="chain",
                hq=32, hkv=8, d=128, window=0, sinks=0, lens=1)
    write = dict(op="append", dtype="bf16", rows=4096, spare=64, pad=7, page=16, hkv=8, d=128)
    commit = dict(op="commit", dtype="bf16", batch=64, nodes=32, hkv=8, d=128)
    return [
        # one new token after a 16k prompt: ordinary decoding, where latency counts
        dict(attn, name="kv4_one_token_16k", nodes=1),
        # the repository's 64k-prefix workload: a 64-node best-first tree
        dict(attn, name="kv4_tree64_64k", prefix_lo=65536, prefix_hi=65536, nodes=64, tree="best"),
        # its ragged batch: 8 sequences of 4k..32k with 32-node trees
        dict(attn, name="kv4_ragged8", batch=8, prefix_lo=4096, prefix_hi=32768, nodes=32, tree="random", lens=4),
        # its largest workload: 128 nodes, 64 query heads, 128k prefix (bound by the products)
        dict(attn, name="kv4_tree128_128k", prefix_lo=131072, prefix_hi=131072, nodes=128, tree="best", hq=64),
        # a windowed layer of a half-precision model with small heads, ragged and odd sizes
        dict(attn, name="kv4_window_d64", dtype="fp16", batch=24, prefix_lo=0, prefix_hi=6001, nodes=17,
             tree="random", hq=16, hkv=2, d=64, window=1000, sinks=4, lens=9),
        # a draft-style window of 512 with the first four positions kept, a chain of 8
        dict(attn, name="window_chain_512", op="window", window=512, sinks=4),
        # a serving batch of a windowed layer: 32 sequences, window 4096
        dict(attn, name="window_batch32_4k", op="window", dtype="fp16", batch=32, prefix_lo=1000, prefix_hi=32768,
             nodes=32, tree="random", window=4096, sinks=4, lens=3),
        # single precision, small heads, odd sizes, a window that some prefixes do not fill
        dict(attn, name="window_fp32_odd", op="window", dtype="fp32", batch=5, prefix_lo=0, prefix_hi=3001, nodes=13,
             tree="random", hq=12, hkv=4, d=64, window=777, sinks=5, lens=6),
        # a prompt of 32k rows written after prefill into a paged cache, and read back
        dict(write, name="append_prompt_32k", rows=32768, spare=1024, pad=0),
        # a batch of decoding steps: one row for each of 200 sequences, some of them padding
        dict(write, name="append_rows_fp32_d64", dtype="fp32", rows=200, hkv=2, d=64),
        # the commit after a verification step of 64 sequences with 32-node trees
        dict(commit, name="commit_batch64"),
        # three sequences, small heads, half precision
        dict(commit, name="commit_three_fp16", dtype="fp16", batch=3, nodes=9, hkv=3, d=64),
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["kv4", "kv4", "window", "window", "append", "commit"])
    d = rng.choice([64, 128])
    if op == "append":
        rows = _log(rng, 1, 32768)
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), rows=rows, spare=rng.randrange(0, 300),
                    pad=rng.choice([0, 0, 3, 11]), page=rng.choice([1, 16, 64]), hkv=rng.choice([1, 2, 3, 8]), d=d)
    if op == "commit":
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), batch=_log(rng, 1, 128), nodes=_log(rng, 1, 128),
                    hkv=rng.choice([1, 2, 5, 8]), d=d)
    hq, hkv = rng.choice([(4, 1), (8, 8), (16, 2), (12, 4), (32, 8), (64, 8)])
    dtype = rng.choice(["bf16", "bf16", "fp16"] if op == "kv4" else ["bf16", "fp16", "fp32"])
    nodes, batch = _log(rng, 1, 128), _log(rng, 1, 32)
    hi = _log(rng, 1, 131072 if dtype != "fp32" else 16384)
    hi = max(1, min(hi, 262144 // batch, int(1.0e9 / (batch * hq * nodes))))
    lo = rng.choice([0, hi // 8, hi // 2, hi])
    window = _log(rng, 1, 16384) if op == "window" or rng.random() < 0.4 else 0
    sinks = rng.choice([0, 1, 4, 130]) if window else 0
    return dict(op=op, dtype=dtype, batch=batch, prefix_lo=lo, prefix_hi=hi, nodes=nodes,
                tree=rng.choice(["chain", "best", "random"]), hq=hq, hkv=hkv, d=d, window=window, sinks=sinks,
                lens=rng.randrange(1000))


def _lengths(case):
    """The prefix length and tree size of each sequence (of the case, not of the seed)."""
    r = random.Random(case["lens"])
    P = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["batch"])]
    return P, [case["nodes"]] * case["batch"]


def _seen(case, P):
    """(first sinks, first key of the window): the prefix keys that a root node sees are
    [0, first) and [second, P)."""
    if not case["window"]:
        return 0, 0
    lo, sk = max(0, P - case["window"] + 1), min(case["sinks"], P)
    return (0, 0) if lo <= sk else (sk, lo)


def _record(d):
    return (9 * d // 8 + 15) // 16 * 16


def work(case):
    d, hkv = case["d"], case["hkv"]
    size = 4 if case["dtype"] == "fp32" else 2
    head = 9 * d // 8                                   # bytes of one row's codes and scales of one head
    if case["op"] == "append":
        written = sum(1 for i in range(case["rows"]) if not _padding(case, i))
        total = case["rows"] + case["spare"]
        # the rows in, their records out; then the cache's records in, their values out
        return {"bytes": written * hkv * (2 * d * size + head) + total * hkv * (head + 2 * d * size),
                "flops": (written * 3 + total) * 2 * d * hkv}
    if case["op"] == "commit":
        rows = case["batch"] * case["nodes"]
        written = sum(_accepted(case, b) for b in range(case["batch"]))
        return {"bytes": written * hkv * (2 * d * size + head) + rows * hkv * (head + 2 * d * size),
                "flops": (written * 3 + rows) * 2 * d * hkv}
    P, m = _lengths(case)
    keys = sum(p - lo + sk for p, (sk, lo) in ((p, _seen(case, p)) for p in P))
    pairs = sum((p - lo + sk + 1) * n for p, n, (sk, lo) in ((p, n, _seen(case, p)) for p, n in zip(P, m)))
    cache = keys * hkv * (head if case["op"] == "kv4" else 2 * d * size)
    nodes = sum(m) * (2 * case["hq"] * d * size + 4 * case["hq"] + 2 * hkv * d * size)
    return {"bytes": cache + nodes, "flops": 4 * d * case["hq"] * pairs}


# ------------------------------------------------------------------------ the inputs

def _parents(r, kind, m):
    """Topologically ordered parent ids of one draft tree (-1: child of the prefix end)."""
    if kind == "chain":
        return list(range(-1, m - 1))
    if kind == "best":  # grown best first: likely nodes get most of the children
        score, parent = [], []
        for i in range(m):
            j = max(range(-1, i), key=lambda a: (0.0 if a < 0 else score[a]) + math.log(r.random()))
            parent.append(j)
            score.append((0.0 if j < 0 else score[j]) - 0.5 * r.random())
        return parent
    return [r.randrange(-1, i) if i else -1 for i in range(m)]


def _accepted(case, b):
    """How many nodes of sequence b the target accepted (of the case, not of the seed)."""
    return random.Random(1000 * b + case["nodes"]).randint(0, min(case["nodes"], 8))


def _padding(case, i):
    return case["pad"] > 0 and i % case["pad"] == case["pad"] - 1


def _rows(g, n, hkv, d):
    """K or V rows as layers make them: normal values, some channels far larger than the rest."""
    x = torch.randn(n, hkv, d, generator=g, device="cuda")
    x[:, :, :: 37] *= 6.0
    return x


def _pack(k, v):
    """The records of rows k, v [n, hkv, d] (values of any floating type), by the module's rule."""
    n, hkv, d = k.shape
    rec = torch.zeros(n, hkv, _record(d), dtype=torch.uint8, device=k.device)
    for at, x in ((0, k), (1, v)):
        s, q = _quantise(x)
        code = (q + 8).to(torch.uint8).view(n, hkv, d // 8, 4, 2).transpose(-1, -2).reshape(n, hkv, d // 2, 2)
        rec[:, :, at * d // 2:(at + 1) * d // 2] = code[..., 0] | (code[..., 1] << 4)
        rec[:, :, d + at * d // 16:d + (at + 1) * d // 16] = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    return rec


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dt, d, hkv = DTYPES[case["dtype"]], case["d"], case["hkv"]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=dict(case), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "append":
        n, total = case["rows"], case["rows"] + case["spare"]
        s["k"], s["v"] = _rows(g, n, hkv, d).to(dt), _rows(g, n, hkv, d).to(dt)
        # the rows' places: pages of the cache in no order
        pages = list(range(total // case["page"] + (total % case["page"] > 0)))
        r.shuffle(pages)
        places = [p * case["page"] + i for p in pages for i in range(case["page"]) if p * case["page"] + i < total]
        s["slot"] = i32([-1 if _padding(case, i) else places[i] for i in range(n)])
        s["cache"] = _pack(_rows(g, total, hkv, d), _rows(g, total, hkv, d))
        return s
    if case["op"] == "commit":
        B, m = case["batch"], case["nodes"]
        s["tree_k"], s["tree_v"] = _rows(g, B * m, hkv, d).to(dt), _rows(g, B * m, hkv, d).to(dt)
        length, path, free = [], [], []
        for b in range(B):
            L = _accepted(case, b)
            length.append(L)
            path += sorted(r.sample(range(m), L)) + [-1] * (m - L)
            free.append(b * m + r.randint(0, m - L))
        s["cu_nodes"], s["accept_len"], s["accept_path"] = i32(list(range(0, B * m + 1, m))), i32(length), i32(path)
        s["dst_row"] = i32(free)
        s["cache"] = _pack(_rows(g, B * m, hkv, d), _rows(g, B * m, hkv, d))
        return s
    P, m = _lengths(case)
    N, rows = sum(m), sum(P)
    cu = lambda a: [sum(a[:i]) for i in range(len(a) + 1)]  # noqa: E731
    s["cu_prefix"], s["cu_nodes"] = i32(cu(P)), i32(cu(m))
    s["parent"] = i32([p for n in m for p in _parents(r, case["tree"], n)])
    s["q"] = torch.randn(N, case["hq"], d, generator=g, device="cuda").to(dt)
    s["tree_k"], s["tree_v"] = _rows(g, N, hkv, d).to(dt), _rows(g, N, hkv, d).to(dt)
    s["max_prefix"], s["max_nodes"] = max(P), max(m)
    s["room"] = max(p - lo + sk for p, (sk, lo) in ((p, _seen(case, p)) for p in P))  # keys that the fullest sequence sees
    k, v = _rows(g, max(1, rows), hkv, d), _rows(g, max(1, rows), hkv, d)
    if case["op"] == "kv4":
        s["cache"] = _pack(k, v)
    else:
        s["k_cache"], s["v_cache"] = k.to(dt), v.to(dt)
    return s


# -------------------------------------------------------------------- the plain forms

def _quantise(x):
    """(scales [..., d / 16], whole multiples [..., d]) of x, decided in 64 bits: values next to a border."""
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=math.inf, neginf=-math.inf)
    x = x.reshape(*x.shape[:-1], -1, 16)
    t = x.abs().amax(-1)
    t = t / torch.full_like(t, 7)  # a true division: one by a number is a product with its reciprocal
    e = torch.frexp(t).exponent.long() - 1
    step = ((e.clamp(-14, 16) - 3 + 1023) << 52).view(torch.float64)  # 2 to that power, exactly
    s = torch.clamp(torch.round(t / step) * step, max=SCALE_MAX)
    q = torch.where(s[..., None] > 0, torch.round(x / s[..., None]), torch.zeros_like(x)).clamp(-7, 7)
    return s, q.reshape(*q.shape[:-2], -1)


def _values(rec, d):
    """The K and V values (32 bits) that records [..., record] stand for."""
    byte = rec[..., :d].reshape(*rec.shape[:-1], d // 4, 4)
    q = torch.stack((byte & 15, byte >> 4), -1).reshape(*byte.shape[:-1], 2, 4).transpose(-1, -2)
    s = (rec[..., d:d + d // 8].to(torch.int16) << 7).view(torch.float16).float()
    x = (q.reshape(*rec.shape[:-1], d // 8, 16).float() - 8) * s[..., None]
    x = x.reshape(*rec.shape[:-1], 2, d)
    return x[..., 0, :], x[..., 1, :]


def _attend(s):
    c, dev = s["case"], s["q"].device
    d, hkv, hq, W, S = c["d"], c["hkv"], c["hq"], c["window"], c["sinks"]
    B, G, n, m = c["batch"], hq // hkv, s["room"], s["max_nodes"]
    p0, n0 = s["cu_prefix"][:-1].long(), s["cu_nodes"][:-1].long()
    P, M = s["cu_prefix"][1:] - p0, s["cu_nodes"][1:] - n0
    # the prefix keys that some node sees: [0, first) and [low, P)
    low = (P - W + 1).clamp(min=0) if W else torch.zeros_like(P)
    first = P.clamp(max=S)
    apart = low > first
    low, first = torch.where(apart, low, 0), torch.where(apart, first, 0)
    j = torch.arange(n, device=dev)
    pos = torch.where(j < first[:, None], j, low[:, None] + j - first[:, None])
    there = pos < P[:, None]
    row = p0[:, None] + torch.where(there, pos, 0)
    if c["op"] == "kv4":
        k, v = _values(s["cache"][row.clamp(max=s["cache"].shape[0] - 1)], d)
    else:
        row = row.clamp(max=s["k_cache"].shape[0] - 1)
        k, v = s["k_cache"][row].float(), s["v_cache"][row].float()
    # the trees: ancestors-or-self from the parents, (I - A)^-1 of the parent matrix
    i = torch.arange(m, device=dev)
    node = (n0[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    live = i < M[:, None]
    parent = torch.where(live, s["parent"][node].long(), -1)
    eye = torch.eye(m, dtype=torch.float64, device=dev).expand(B, m, m)
    edge = (parent[:, :, None] == i).double()
    anc = torch.linalg.solve_triangular(eye - edge, eye, upper=False, unitriangular=True) > 0.5
    depth = anc.sum(-1) - 1
    t = P[:, None] + depth
    sees = there[:, None, :].expand(B, m, n)
    if W:
        sees = sees & ((t[:, :, None] - pos[:, None, :] < W) | (pos[:, None, :] < S))
        anc = anc & ((t[:, :, None] - t[:, None, :] < W) | (t[:, None, :] < S))
    sees = torch.cat((sees, anc & live[:, None, :]), -1)
    k = torch.cat((k, s["tree_k"][node].float()), 1).permute(0, 2, 3, 1)
    v = torch.cat((v, s["tree_v"][node].float()), 1).permute(0, 2, 1, 3)
    q = s["q"][node].float().view(B, m, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, m * G, d)
    z = torch.matmul(q * (1.0 / math.sqrt(d)), k).view(B, hkv, m, G, n + m)
    z.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, hkv, m * G, n + m), v).view(B, hkv, m, G, d) / total
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, m, hq, d)[live]
    lse = lse.permute(0, 2, 1, 3).reshape(B, m, hq)[live]
    return {"out": o.to(s["q"].dtype), "lse": lse}


def _overlay(s, row, k, v):
    """The cache's values with k, v [n, hkv, d] quantised into rows `row` (-1: not written)."""
    d, rows = s["case"]["d"], s["cache"].shape[0]
    dt = k.dtype
    outs = []
    for old, x in zip(_values(s["cache"], d), (k, v)):
        scale, q = _quantise(x)
        new = (q.view(*scale.shape, 16) * scale[..., None]).float().reshape(x.shape)
        old = torch.cat((old, torch.zeros_like(old[:1])))
        old[torch.where(row < 0, rows, row).long()] = new
        outs.append(old[:rows].to(dt))
    return {"k": outs[0], "v": outs[1]}


def run(state):
    s = state
    c = s["case"]
    if own:
        from tree_verification_attention_gb300 import api
        if c["op"] == "append":
            api.append_kv4(s["k"], s["v"], s["slot"], s["cache"], dev_status=s["status"])
            k, v = api.read_kv4(s["cache"], c["d"], dtype=s["k"].dtype, dev_status=s["status"])
            return {"k": k, "v": v}
        if c["op"] == "commit":
            api.commit_accepted_kv4(s["cu_nodes"], s["accept_len"], s["accept_path"], s["tree_k"], s["tree_v"],
                                    s["dst_row"], s["cache"], max_nodes=c["nodes"], dev_status=s["status"])
            k, v = api.read_kv4(s["cache"], c["d"], dtype=s["tree_k"].dtype, dev_status=s["status"])
            return {"k": k, "v": v}
        if s.get("params") is None:  # the caller's plan: made at its first step, kept for the later ones
            cache = s["cache"] if c["op"] == "kv4" else s["k_cache"]
            s["params"] = api.make_params(s["q"], cache, s["cu_prefix"], s["cu_nodes"], c["hkv"], s["max_prefix"],
                                          s["max_nodes"])
            s["workspace"] = api.alloc_workspace(s["params"], s["q"].device)
        if c["op"] == "kv4":
            out, lse = api.tree_verify_attn_kv4_varlen(
                s["q"], s["cache"], s["tree_k"], s["tree_v"], s["parent"], s["cu_prefix"], s["cu_nodes"],
                s["max_prefix"], s["max_nodes"], window=c["window"], sinks=c["sinks"], workspace=s["workspace"],
                dev_status=s["status"], params=s["params"])
        else:
            out, lse = api.tree_verify_attn_window_varlen(
                s["q"], s["k_cache"], s["v_cache"], s["tree_k"], s["tree_v"], s["parent"], s["cu_prefix"],
                s["cu_nodes"], s["max_prefix"], s["max_nodes"], window=c["window"], sinks=c["sinks"],
                workspace=s["workspace"], dev_status=s["status"], params=s["params"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        return _overlay(s, s["slot"], s["k"], s["v"])
    if c["op"] == "commit":
        j = torch.arange(c["nodes"], device=s["slot"].device if "slot" in s else s["accept_len"].device)
        taken = j < s["accept_len"][:, None]
        node = s["cu_nodes"][:-1, None] + torch.where(taken, s["accept_path"].view(-1, c["nodes"]), 0)
        row = torch.where(taken, s["dst_row"][:, None] + j, -1).reshape(-1)
        node = node.reshape(-1).long()
        return _overlay(s, row, s["tree_k"][node], s["tree_v"][node])
    return _attend(s)


# ---------------------------------------------------- the definition, written out in 64 bits

def _all_scales():
    """The 256 scale bytes' values, up to the largest that is used."""
    v = [(b % 8) * 2.0 ** -17 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 15) for b in range(256)]
    return torch.tensor([x for x in v if x <= SCALE_MAX], dtype=torch.float64, device="cuda")


def _nearest(levels, x):
    """The nearest of ascending `levels` to x, and its number; halfway goes to the even number."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo = torch.searchsorted(mid, x.contiguous(), right=False)  # borders strictly below x
    hi = torch.searchsorted(mid, x.contiguous(), right=True)   # borders at or below x
    at = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    return levels[at], at


def _exact_rows(x):
    x = x.double()
    levels = _all_scales()
    blocks = x.view(x.shape[0], x.shape[1], x.shape[2] // 16, 16)
    biggest = blocks.abs().max(dim=3).values
    scale, _ = _nearest(levels * 7, biggest)
    scale = scale / torch.full_like(scale, 7)
    # numbers -8 .. 8 as levels 0 .. 16: an even level is an even number
    whole = torch.arange(-8, 9, dtype=torch.float64, device=x.device)
    ratio = torch.where(scale[..., None] > 0, blocks / scale[..., None].clamp(min=1e-30), torch.zeros_like(blocks))
    q, _ = _nearest(whole, ratio)
    return (q.clamp(-7, 7) * scale[..., None]).view(x.shape)


def _exact_cache(cache, d):
    table = torch.cat((_all_scales(), torch.zeros(256, dtype=torch.float64, device=cache.device)))
    halves = []
    for at in (0, 1):
        codes = cache[:, :, at * d // 2:(at + 1) * d // 2].long()
        x = torch.zeros(cache.shape[0], cache.shape[1], d, dtype=torch.float64, device=cache.device)
        for e in range(8):  # element 8 i + e: bits 4 (e // 2) + 16 (e % 2) of code word i
            bit = 4 * (e // 2) + 16 * (e % 2)
            x[:, :, e::8] = ((codes[:, :, bit // 8::4] >> (bit % 8)) % 16 - 8).double()
        scale = table[cache[:, :, d + at * d // 16:d + (at + 1) * d // 16].long()]
        halves.append(x * scale.repeat_interleave(16, dim=2))
    return halves


def exact(case, seed):
    s = prepare(case, seed)
    d, hkv = case["d"], case["hkv"]
    if case["op"] in ("append", "commit"):
        k, v = _exact_cache(s["cache"], d)
        if case["op"] == "append":
            pairs = [(i, int(r)) for i, r in enumerate(s["slot"].tolist()) if r >= 0]
            src_k, src_v = s["k"], s["v"]
        else:
            pairs, src_k, src_v = [], s["tree_k"], s["tree_v"]
            path, m = s["accept_path"].tolist(), case["nodes"]
            for b, (L, at) in enumerate(zip(s["accept_len"].tolist(), s["dst_row"].tolist())):
                pairs += [(b * m + path[b * m + j], at + j) for j in range(L)]
        if pairs:
            src, dst = (torch.tensor(a, device=k.device) for a in zip(*pairs))
            k[dst] = _exact_rows(src_k[src])
            v[dst] = _exact_rows(src_v[src])
        return {"k": k, "v": v}
    P, m = _lengths(case)
    hq, W, S = case["hq"], case["window"], case["sinks"]
    G = hq // hkv
    outs, lses, p0, n0 = [], [], 0, 0
    for b in range(case["batch"]):
        par = s["parent"][n0:n0 + m[b]].tolist()
        anc, depth = [], []
        for i in range(m[b]):
            up, a = [], i
            while a >= 0:
                up.append(a)
                a = par[a]
            anc.append(up)
            depth.append(len(up) - 1)
        at = [P[b] + x for x in depth]  # the nodes' positions
        sk, lo = _seen(case, P[b])
        keys = list(range(0, sk)) + list(range(lo, P[b]))
        pos = torch.tensor(keys, dtype=torch.long, device="cuda")
        t = torch.tensor(at, device="cuda")
        see = torch.ones(m[b], len(keys), dtype=torch.bool, device="cuda")
        if W:
            see = (t[:, None] - pos[None, :] < W) | (pos[None, :] < S)
        tree = torch.zeros(m[b], m[b], dtype=torch.bool)
        for i in range(m[b]):
            for a in anc[i]:
                tree[i, a] = not W or at[i] - at[a] < W or at[a] < S
        see = torch.cat((see, tree.cuda()), 1).repeat_interleave(G, 0)
        if case["op"] == "kv4":
            pk, pv = _exact_cache(s["cache"][p0 + pos], d)
        else:
            pk, pv = s["k_cache"][p0 + pos].double(), s["v_cache"][p0 + pos].double()
        o = torch.empty(m[b], hq, d, dtype=torch.float64, device="cuda")
        L = torch.empty(m[b], hq, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            kk = torch.cat((pk[:, h], s["tree_k"][n0:n0 + m[b], h].double()))
            vv = torch.cat((pv[:, h], s["tree_v"][n0:n0 + m[b], h].double()))
            qq = s["q"][n0:n0 + m[b], h * G:(h + 1) * G].double().reshape(m[b] * G, d)
            z = torch.where(see, qq @ kk.T / math.sqrt(d), torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
            l = torch.logsumexp(z, 1)
            o[:, h * G:(h + 1) * G] = (torch.exp(z - l[:, None]) @ vv).view(m[b], G, d)
            L[:, h * G:(h + 1) * G] = l.view(m[b], G)
        outs.append(o)
        lses.append(L)
        p0, n0 = p0 + P[b], n0 + m[b]
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
