"""The measured cases of the Gated DeltaNet state operators and of cross attention.

Three operators, reached through ``tree_verification_attention_gb300.api``:

* ``gdn_update_varlen``: every sequence's tokens through a Gated DeltaNet layer's rule,

      S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t,

  from its committed state, which is updated in place: single tokens of ordinary decoding,
  whole prompts, and ragged mixtures of both;
* ``commit_accepted_gdn``: the same update of the state along the accepted path of a draft
  tree (what ``gdn_tree_verify`` leaves to the commit);
* ``cross_attn_varlen``: every query of a sequence attends to all keys of a cache of another
  length, without a mask: a draft model's cross-attention onto the target's K/V cache.
  Without a key the output is 0 and the log-sum-exp -infinity.

Each case is a plain dict; the comments in ``listed`` say what it stands for.
"""
import math
import random

import torch

own = False  # True: run() calls the framework's operators; False: their plain form

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 64  # tokens that the plain form takes at a time


# ------------------------------------------------------------------------- the cases

def listed():
    gdn = dict(op="gdn", dtype="bf16", batch=1, len_lo=1, len_hi=1, heads=32, d=128, fresh=False, lens=1)
    commit = dict(op="commit", dtype="bf16", batch=64, nodes=32, heads=32, d=128)
    cross = dict(op="cross", dtype="bf16", batch=1, keys_lo=32768, keys_hi=32768, queries=16, hq=32, hkv=8, d=128,
                 lens=1)
    return [
        # one new token of one sequence: ordinary decoding, where latency counts
        dict(gdn, name="gdn_one_token"),
        # a decoding step of a serving batch: 64 sequences, a token each
        dict(gdn, name="gdn_tokens_batch64", batch=64),
        # a prompt of 4k tokens from an empty state
        dict(gdn, name="gdn_prompt_4k", len_lo=4096, len_hi=4096, fresh=True),
        # the longest prompt of the repository's prefix lengths below 64k: 32k tokens
        dict(gdn, name="gdn_prompt_32k", len_lo=32768, len_hi=32768, fresh=True),
        # a ragged batch with small heads: prompts and continued prompts of odd lengths
        dict(gdn, name="gdn_ragged_d64", batch=24, len_lo=1, len_hi=2001, heads=16, d=64, lens=5),
        # single precision, odd lengths, empty sequences among them
        dict(gdn, name="gdn_fp32_odd", dtype="fp32", batch=5, len_lo=0, len_hi=777, heads=6, lens=8),
        # the commit after a verification step of 64 sequences with 32-node trees
        dict(commit, name="commit_gdn_batch64"),
        # three sequences, few small heads, single precision
        dict(commit, name="commit_gdn_three_fp32", dtype="fp32", batch=3, nodes=9, heads=4, d=64),
        # one step of a beam of 16 drafts over a 32k prompt, LongSpec's own precision
        dict(cross, name="cross_beam16_32k", dtype="fp16"),
        # one draft token of each of 8 sequences, prefixes of 4k to 32k
        dict(cross, name="cross_ragged8", batch=8, keys_lo=4096, keys_hi=32768, queries=1, lens=4),
        # a long run of queries over a middling cache (bound by the products), odd sizes
        dict(cross, name="cross_2001_queries", keys_lo=8190, keys_hi=8190, queries=2001),
        # single precision, small heads, odd sizes, sequences without keys among them
        dict(cross, name="cross_fp32_odd", dtype="fp32", batch=6, keys_lo=0, keys_hi=3001, queries=13, hq=12, hkv=4,
             d=64, lens=9),
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gdn", "gdn", "gdn", "commit", "cross", "cross"])
    d = rng.choice([64, 128])
    if op == "commit":
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), batch=_log(rng, 1, 64), nodes=_log(rng, 1, 128),
                    heads=rng.choice([1, 3, 8, 16, 32]), d=d)
    if op == "gdn":
        dtype, heads = rng.choice(["bf16", "bf16", "fp32"]), rng.choice([1, 2, 5, 16, 32])
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 32768 if dtype == "bf16" else 4096)
        hi = max(1, min(hi, 32768 * 32 // (batch * heads)))
        return dict(op=op, dtype=dtype, batch=batch, len_lo=rng.choice([0, hi // 3, hi]), len_hi=hi, heads=heads, d=d,
                    fresh=rng.random() < 0.5, lens=rng.randrange(1000))
    hq, hkv = rng.choice([(4, 1), (8, 8), (16, 2), (12, 4), (32, 8), (64, 8)])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    queries, batch = _log(rng, 1, 2048 if dtype != "fp32" else 64), _log(rng, 1, 32)
    hi = _log(rng, 1, 65536 if dtype != "fp32" else 8192)
    hi = max(1, min(hi, 262144 // batch, int(4.0e8 / (batch * hq * queries))))
    return dict(op=op, dtype=dtype, batch=batch, keys_lo=rng.choice([0, hi // 8, hi // 2, hi]), keys_hi=hi,
                queries=queries, hq=hq, hkv=hkv, d=d, lens=rng.randrange(1000))


def _lengths(case):
    """Each sequence's tokens or keys (of the case, not of the seed)."""
    r = random.Random(case["lens"])
    lo, hi = (case["len_lo"], case["len_hi"]) if case["op"] == "gdn" else (case["keys_lo"], case["keys_hi"])
    n = [r.randint(lo, hi) for _ in range(case["batch"])]
    if lo == 0 and len(n) > 1:
        n[1] = 0
    if not any(n):
        n[0] = hi
    return n


def _accepted(case, b):
    """How many nodes of sequence b the target accepted (of the case, not of the seed)."""
    return random.Random(1000 * b + case["nodes"]).randint(1 if b == 0 else 0, min(case["nodes"], 8))


def work(case):
    d, size = case["d"], 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "cross":
        P, m, hq, hkv = _lengths(case), case["queries"], case["hq"], case["hkv"]
        # K and V once, each query in, its output and log-sum-exp out
        return {"bytes": sum(P) * 2 * hkv * d * size + len(P) * m * hq * (2 * d * size + 4),
                "flops": 4 * d * hq * m * sum(P)}
    H = case["heads"]
    if case["op"] == "gdn":
        n, moves, products = _lengths(case), 4, 6   # q, k, v in, the output out; K.S, Q.S and the update
    else:
        n, moves, products = [_accepted(case, b) for b in range(case["batch"])], 2, 4
    states = sum(1 for x in n if x)
    return {"bytes": sum(n) * H * (moves * d * size + 8) + states * 2 * H * d * d * 4,
            "flops": sum(n) * H * products * d * d}


# ------------------------------------------------------------------------ the inputs

def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _layer(g, n, H, d, dt):
    """q, k, v, beta and alpha of n tokens as a Gated DeltaNet layer makes them: unit keys, queries
    scaled by d^-1/2, write strengths in (0, 1), decays from heads that forget in a few tokens to
    heads that keep hundreds."""
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rate = torch.exp(torch.linspace(math.log(0.003), math.log(0.5), H, device="cuda"))
    return dict(q=(_unit(r(n, H, d)) * d ** -0.5).to(dt), k=_unit(r(n, H, d)).to(dt), v=r(n, H, d).to(dt),
                beta=torch.sigmoid(r(n, H)), alpha=torch.exp(-rate * torch.nn.functional.softplus(r(n, H))))


def _states(g, B, H, d):
    """States that have absorbed some context."""
    return 0.3 * torch.randn(B, H, d, d, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    dt, d, B = DTYPES[case["dtype"]], case["d"], case["batch"]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = lambda a: i32([sum(a[:i]) for i in range(len(a) + 1)])  # noqa: E731
    s = dict(case=dict(case), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "gdn":
        n, H = _lengths(case), case["heads"]
        s.update(_layer(g, sum(n), H, d, dt), cu_tokens=cu(n), max_tokens=max(n))
        s["state"] = _states(g, B, H, d)
        if case["fresh"]:
            s["state"].zero_()
        return s
    if case["op"] == "commit":
        m, H = case["nodes"], case["heads"]
        s.update(_layer(g, B * m, H, d, dt), state=_states(g, B, H, d), cu_nodes=cu([m] * B))
        length, path = [_accepted(case, b) for b in range(B)], []
        for L in length:
            path += sorted(r.sample(range(m), L)) + [-1] * (m - L)
        s["accept_len"], s["accept_path"], s["longest"] = i32(length), i32(path), max(length)
        return s
    P, m, hkv = _lengths(case), case["queries"], case["hkv"]
    rows = lambda n, h: torch.randn(n, h, d, generator=g, device="cuda")  # noqa: E731
    k, v = rows(max(1, sum(P)), hkv), rows(max(1, sum(P)), hkv)
    k[:, :, ::37] *= 3.0  # some channels larger than the rest
    s.update(q=rows(B * m, case["hq"]).to(dt), k_cache=k.to(dt), v_cache=v.to(dt), cu_keys=cu(P),
             cu_queries=cu([m] * B), max_keys=max(P))
    return s


# -------------------------------------------------------------------- the plain forms

def _padded(cu, longest, rows):
    """Row numbers [B, longest] of ragged sequences, and which of them exist."""
    j = torch.arange(longest, device=cu.device)
    first = cu[:-1].long()[:, None]
    live = j < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, first + j, 0).clamp(max=max(0, rows - 1)), live


def _delta_rule(s, row, live, state, want_out):
    """The rule over rows [B, L] (where `live`) in chunks: (outputs [B, L, H, d] or None, new state)."""
    B, L = row.shape
    H, d = s["k"].shape[1:]
    C = min(CHUNK, L)
    n = -(-L // C)
    pad = n * C - L
    row = torch.nn.functional.pad(row, (0, pad))
    live = torch.nn.functional.pad(live, (0, pad))

    def tile(x, empty):  # [B, n C, H, ...] of the rows, as chunks [B, H, n, C, ...]
        x = x[row].float()
        x = torch.where(live.view(live.shape + (1,) * (x.dim() - 2)), x, torch.full_like(x, empty))
        return x.transpose(1, 2).reshape(B, H, n, C, *x.shape[3:])

    k, v, b, a = tile(s["k"], 0.0), tile(s["v"], 0.0), tile(s["beta"], 0.0), tile(s["alpha"], 1.0)
    c = a.double().log().cumsum(-1)
    lower = torch.ones(C, C, dtype=torch.bool, device=row.device).tril()
    ratio = torch.where(lower, (c[..., :, None] - c[..., None, :]).masked_fill(~lower, 0.0).exp(), 0.0).float()
    start, end = c.exp().float(), (c[..., -1:] - c).exp().float()  # from the chunk's start; to its end
    kk = torch.matmul(k, k.transpose(-1, -2))
    A = (b[..., None] * ratio * kk).tril(-1)
    eye = torch.eye(C, device=row.device)
    T = torch.linalg.solve_triangular(eye + A, eye.expand_as(A), upper=False, unitriangular=True) * b[..., None, :]
    del A, kk
    if want_out:
        q = tile(s["q"], 0.0)
        inner = ratio * torch.matmul(q, k.transpose(-1, -2))
    S, outs = state, []
    for i in range(n):
        U = torch.matmul(T[:, :, i], v[:, :, i] - start[:, :, i, :, None] * torch.matmul(k[:, :, i], S))
        if want_out:
            outs.append(start[:, :, i, :, None] * torch.matmul(q[:, :, i], S) + torch.matmul(inner[:, :, i], U))
        S = start[:, :, i, -1, None, None] * S + torch.matmul((end[:, :, i, :, None] * k[:, :, i]).transpose(-1, -2), U)
    out = torch.cat(outs, 2).transpose(1, 2)[:, :L] if want_out else None
    return out, S


def _cross(s):
    c, B, m, hkv, hq, d = (s["case"], *(s["case"][x] for x in ("batch", "queries", "hkv", "hq", "d")))
    G = hq // hkv
    row, there = _padded(s["cu_keys"], max(1, s["max_keys"]), s["k_cache"].shape[0])
    k = s["k_cache"][row].float().permute(0, 2, 3, 1)
    v = torch.where(there[:, :, None, None], s["v_cache"][row].float(), 0.0).permute(0, 2, 1, 3)
    q = s["q"].float().view(B, m, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, m * G, d)
    z = torch.matmul(q * (1.0 / math.sqrt(d)), k)
    z.masked_fill_(~there[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    o = o.view(B, hkv, m, G, d).permute(0, 2, 1, 3, 4).reshape(B * m, hq, d)
    return {"out": o.to(s["q"].dtype), "lse": lse.view(B, hkv, m, G).permute(0, 2, 1, 3).reshape(B * m, hq)}


def run(state):
    s = state
    c = s["case"]
    if own:
        from tree_verification_attention_gb300 import api
        if c["op"] == "gdn":
            out = api.gdn_update_varlen(s["q"], s["k"], s["v"], s["beta"], s["alpha"], s["cu_tokens"], s["max_tokens"],
                                        s["state"], dev_status=s["status"])
            return {"out": out, "state": s["state"]}
        if c["op"] == "commit":
            api.commit_accepted_gdn(s["cu_nodes"], s["accept_len"], s["accept_path"], s["k"], s["v"], s["beta"],
                                    s["alpha"], s["state"], max_nodes=c["nodes"], dev_status=s["status"])
            return {"state": s["state"]}
        if s.get("params") is None:  # the caller's plan: made at its first step, kept for the later ones
            s["params"] = api.make_params(s["q"], s["k_cache"], s["cu_keys"], s["cu_queries"], c["hkv"], s["max_keys"],
                                          c["queries"])
            s["workspace"] = api.alloc_cross_workspace(s["params"], s["q"].device)
        out, lse = api.cross_attn_varlen(s["q"], s["k_cache"], s["v_cache"], s["cu_queries"], s["cu_keys"],
                                         c["queries"], s["max_keys"], workspace=s["workspace"],
                                         dev_status=s["status"], params=s["params"])
        return {"out": out, "lse": lse}
    if c["op"] == "gdn":
        row, live = _padded(s["cu_tokens"], s["max_tokens"], s["k"].shape[0])
        out, S = _delta_rule(s, row, live, s["state"], True)
        s["state"].copy_(S)
        return {"out": out[live].to(s["q"].dtype), "state": s["state"]}
    if c["op"] == "commit":
        live = torch.arange(s["longest"], device=s["state"].device) < s["accept_len"][:, None]
        path = s["accept_path"].view(c["batch"], c["nodes"])[:, :s["longest"]]
        row = torch.where(live, s["cu_nodes"][:-1, None] + path, 0).long()
        s["state"].copy_(_delta_rule(s, row, live, s["state"], False)[1])
        return {"state": s["state"]}
    return _cross(s)


# ---------------------------------------------------- the definition, written out in 64 bits

def _token_by_token(s, rows, want_out):
    """The recurrence itself: `rows` holds each sequence's row numbers, first token first."""
    S = s["state"].double()
    H, d = s["k"].shape[1:]
    outs = torch.zeros(s["k"].shape[0], H, d, dtype=torch.float64, device="cuda") if want_out else None
    by_length = sorted(range(len(rows)), key=lambda b: -len(rows[b]))
    longest = len(rows[by_length[0]])
    table = torch.zeros(len(rows), longest, dtype=torch.long)
    for i, b in enumerate(by_length):
        table[i, :len(rows[b])] = torch.tensor(rows[b], dtype=torch.long)
    table = table.cuda()
    work = S[torch.tensor(by_length, device="cuda")].clone()
    counts = [len(rows[b]) for b in by_length]
    many = len(rows)
    for t in range(longest):
        while counts[many - 1] <= t:  # the longest sequences come first
            many -= 1
        at = table[:many, t]
        k, v = s["k"][at].double(), s["v"][at].double()
        a, b = s["alpha"][at].double()[..., None], s["beta"][at].double()[..., None]
        now = work[:many]
        read = (now * k[..., :, None]).sum(2)
        now.mul_(a[..., None]).add_(k[..., :, None] * (b * (v - a * read))[..., None, :])
        if want_out:
            outs[at] = (now * s["q"][at].double()[..., :, None]).sum(2)
    S[torch.tensor(by_length, device="cuda")] = work
    return outs, S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gdn":
        rows, first = [], 0
        for n in _lengths(case):
            rows.append(list(range(first, first + n)))
            first += n
        out, S = _token_by_token(s, rows, True)
        return {"out": out, "state": S}
    if case["op"] == "commit":
        m, path = case["nodes"], s["accept_path"].tolist()
        rows = [[b * m + path[b * m + j] for j in range(L)] for b, L in enumerate(s["accept_len"].tolist())]
        return {"state": _token_by_token(s, rows, False)[1]}
    P, m, hq, hkv, d = _lengths(case), case["queries"], case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    out = torch.zeros(len(P) * m, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((len(P) * m, hq), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, p in enumerate(P):
        mine = slice(b * m, (b + 1) * m)
        for h in range(hq if p else 0):
            kk, vv = s["k_cache"][first:first + p, h // G].double(), s["v_cache"][first:first + p, h // G].double()
            z = s["q"][mine, h].double() @ kk.T / math.sqrt(d)
            l = torch.logsumexp(z, 1)
            out[mine, h] = torch.exp(z - l[:, None]) @ vv
            lse[mine, h] = l
        first += p
    return {"out": out, "lse": lse}
