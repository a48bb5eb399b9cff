"""Helpers for the Gated DeltaNet update and commit tests: cases on the device, and the recurrence in
float64 written with torch (for sequences too long for the oracle's loops; pinned to it on the CPU).

Bars.  Keys and queries are unit vectors, beta in (0, 1), alpha <= 1, so a step never enlarges a
column of the state; columns have norms M of a few units (8 at most here).
* float32: a step's dot products over d rows are off by some sqrt(d) 2^-24 M (3e-7 M; d 2^-24 M =
  6e-5 if every rounding fell the same way), and the decay keeps some 15 steps' worth: a few 1e-6
  to 1e-5.  Bar: 2e-4 + 1e-4 |ref|, as for gdn_tree_verify, and 1e-5 of the whole in the 2-norm.
* bf16 states: every operand of a product is held to 16 bits or more, so a term is off by at most
  2^-17 on each side: at most 2^-16 M = 1.2e-4 a dot if all fell the same way, and like
  2^-17 M / sqrt(d) otherwise.  The same bars.
* bf16 outputs: one rounding of the result (2^-8 |ref|) and, in the chunked form, the matrix of
  products inside a chunk and the corrections it multiplies in bf16, rounded 4 times in all
  (2^-8 each) before the sum over up to 64 tokens whose terms are about 2^-3.5 each (q.k of unit
  vectors in 128 dimensions times values of size 1): sqrt(64) 2^-3.5 sqrt(4) 2^-8 / sqrt(3) = 3e-3 as
  a standard deviation for v of size 1, times up to 2 for d = 64 and larger values.  Bars: 5e-3 of the
  whole in the 2-norm, and 0.04 + 2^-8 |ref| (over 5 deviations) for each value.  Calls whose
  longest sequence is short take the recurrence: 2e-4 + (1e-4 + 2^-8) |ref|."""
import numpy as np
import torch

from tree_verification_attention_gb300 import api, workloads

SHORT = 16  # bf16 calls of at most so many tokens a sequence: the recurrence


def case(lens, heads=2, d=64, dtype="fp32", seed=0, **kw):
    return workloads.make_gdn_case(batch=len(lens), heads=heads, d=d, seed=seed, dtype=dtype,
                                   parents=[workloads.chain_tree(n) if n else np.zeros(0, np.int64) for n in lens], **kw)


def device(c, dtype, spare=0):
    """The case's tensors, with `spare` rows of NaN behind the last sequence."""
    t = {}
    for n in ("q", "k", "v", "beta", "alpha"):
        x = torch.from_numpy(np.ascontiguousarray(c[n]))
        x = torch.cat([x, torch.full((spare, *x.shape[1:]), float("nan"))]).cuda()
        t[n] = x.to(torch.bfloat16) if dtype == "bf16" and n in "qkv" else x
    t["state"] = torch.from_numpy(c["S0"].copy()).cuda()
    t["cu_tokens"] = torch.from_numpy(c["cu_nodes"]).int().cuda()
    return t


def run(t, max_tokens, out=None, status=0, **kw):
    """(outputs, state) of a call on a copy of the state; the status word has to be `status`."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    S = t["state"].clone()
    out = api.gdn_update_varlen(t["q"], t["k"], t["v"], t["beta"], t["alpha"], t["cu_tokens"], max_tokens, S, out=out,
                                dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return out, S


def recurrence(q, k, v, beta, alpha, cu, state):
    """(outputs, new state) in float64, on the tensors' device."""
    S = state.double().clone()
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    for b in range(len(cu) - 1):
        for t in range(int(cu[b]), int(cu[b + 1])):
            kt, vt = k[t].double(), v[t].double()
            a, be = alpha[t].double()[:, None], beta[t].double()[:, None]
            w = be * (vt - a * (S[b] * kt[:, :, None]).sum(1))
            S[b] = a[:, :, None] * S[b] + kt[:, :, None] * w[:, None, :]
            out[t] = (S[b] * q[t].double()[:, :, None]).sum(1)
    return out, S


def check(out, S, ref, S_ref, dtype, longest):
    """Against float64 at the bars above (rows of the sequences only)."""
    n = ref.shape[0]
    out, S, ref, S_ref = (torch.as_tensor(x).double().cpu() for x in (out[:n], S, ref, S_ref))
    assert torch.isfinite(S).all() and torch.isfinite(out).all()
    err = (S - S_ref).abs()
    assert (err <= 2e-4 + 1e-4 * S_ref.abs()).all(), float(err.max())
    assert (S - S_ref).norm() <= 1e-5 * S_ref.norm() + 1e-30, float((S - S_ref).norm() / S_ref.norm())
    err = (out - ref).abs()
    if dtype == "fp32":
        bar = 2e-4 + 1e-4 * ref.abs()
    elif longest <= SHORT:
        bar = 2e-4 + (1e-4 + 2.0 ** -8) * ref.abs()
    else:
        bar = 0.04 + 2.0 ** -8 * ref.abs()
    assert (err <= bar).all(), float(err.max())
    if n:
        assert (out - ref).norm() <= (1e-5 if dtype == "fp32" else 5e-3) * ref.norm() + 1e-30
