"""ctypes binding over ``libtva.so`` (include/tva.h), with the C entry points' names.

Argument marshalling only: torch tensors provide device memory and the current CUDA
stream; every step of the computation runs in the library's kernels.  There is no
CPU path: if the library is missing or a tensor is not on a CUDA device, the call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

from . import build as _build

__all__ = [
    "TvaError", "Params", "load_library", "workspace_size", "num_workers",
    "tree_verify_attn_varlen", "tree_verify_attn_partials", "tree_verify_attn_combine",
    "tree_verify_attn", "read_device_status", "release", "diag_set_wait_limit", "diag_use_cta_pair", "accept_longest_path",
    "tree_verify_attn_window_varlen", "tree_verify_attn_kv4_varlen", "kv4_record_bytes", "alloc_kv4_cache", "append_kv4",
    "read_kv4", "commit_accepted_kv4", "status_string", "STATUS",
]

STATUS = {0: "TVA_OK", 1: "TVA_ERR_INVALID_ARG", 2: "TVA_ERR_UNSUPPORTED", 3: "TVA_ERR_BAD_TREE",
          4: "TVA_ERR_WORKSPACE", 5: "TVA_ERR_CUDA", 6: "TVA_ERR_TIMEOUT"}
DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


class TvaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


class Params(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("softmax_scale", ctypes.c_float),
        ("cu_prefix", ctypes.c_void_p), ("cu_nodes", ctypes.c_void_p),
        ("max_prefix_len", ctypes.c_int), ("max_nodes", ctypes.c_int),
        ("kv_capacity", ctypes.c_int), ("node_capacity", ctypes.c_int),
    ]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def load_library(path: str | None = None):
    """Load libtva.so (built by ``build.build()``); raises if it is absent.  The
    environment variable TVA_LIBRARY selects another build of the same library (for
    example libtva_checked.so, the index-checked variant)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("TVA_LIBRARY") or _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run tree_verification_attention_gb300.build.build() "
                           "(or __graft_entry__.build()) first; there is no fallback path")
    lib = ctypes.CDLL(path)
    PP = ctypes.POINTER(Params)
    sig = {
        "tva_workspace_size": (_SZ, [PP]),
        "tva_num_workers": (_I, [PP]),
        "tree_verify_attn_varlen": (_I, [PP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
        "tree_verify_attn_partials": (_I, [PP, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
        "tree_verify_attn_combine": (_I, [PP, _P, _SZ, _P, _P, _P, _P]),
        "tree_verify_attn": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
        "tva_read_device_status": (_I, [ctypes.POINTER(ctypes.c_int32), _P]),
        "tva_release": (None, []),
        "tva_diag_set_wait_limit": (None, [ctypes.c_ulonglong, _I]),
        "tva_diag_use_cta_pair": (None, [_I]),
        "accept_longest_path": (_I, [_I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "commit_accepted_kv": (_I, [_I, _I, _I, _I, _I, _I, ctypes.c_longlong, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P]),
        "verify_chain_sampling": (_I, [_I, _I, _I, ctypes.c_longlong, ctypes.c_longlong, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _P]),
        "gdn_tree_verify": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
        "tree_verify_attn_window_varlen": (_I, [PP, _I, _I] + [_P] * 9 + [_SZ, _P, _P]),
        "tree_verify_attn_kv4_varlen": (_I, [PP, _I, _I] + [_P] * 8 + [_SZ, _P, _P]),
        "tva_kv4_record_bytes": (_SZ, [_I]),
        "append_kv4": (_I, [_I, _I, _I, _I, ctypes.c_longlong] + [_P] * 6),
        "read_kv4": (_I, [_I, _I, _I, _I, ctypes.c_longlong] + [_P] * 6),
        "commit_accepted_kv4": (_I, [_I, _I, _I, _I, _I, _I, ctypes.c_longlong] + [_P] * 9),
        "tva_status_string": (ctypes.c_char_p, [_I]),
        "tva_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().tva_status_string(code).decode()


def _check(code: int, where: str):
    if code != 0:
        detail = load_library().tva_last_error().decode() if code == 5 else ""
        raise TvaError(code, where + (f" [{detail}]" if detail else ""))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def make_params(q, k_cache, cu_prefix, cu_nodes, num_kv_heads, max_prefix_len, max_nodes,
                softmax_scale=0.0) -> Params:
    if q.dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}")
    N, Hq, d = q.shape
    return Params(batch=cu_prefix.numel() - 1, num_q_heads=Hq, num_kv_heads=num_kv_heads, head_dim=d,
                  dtype=DTYPES[q.dtype], softmax_scale=float(softmax_scale),
                  cu_prefix=cu_prefix.data_ptr(), cu_nodes=cu_nodes.data_ptr(),
                  max_prefix_len=int(max_prefix_len), max_nodes=int(max_nodes),
                  kv_capacity=k_cache.shape[0], node_capacity=N)


def workspace_size(params: Params) -> int:
    return int(load_library().tva_workspace_size(ctypes.byref(params)))


def num_workers(params: Params) -> int:
    return int(load_library().tva_num_workers(ctypes.byref(params)))


def alloc_workspace(params: Params, device) -> torch.Tensor:
    n = workspace_size(params)
    if n == 0:
        raise TvaError(1, "tva_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _attn_inputs(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes):
    _dev(q, "q")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("tree_k", tree_k), ("tree_v", tree_v)):
        _dev(t, name, q.dtype)
    for name, t in (("parent", parent), ("cu_prefix", cu_prefix), ("cu_nodes", cu_nodes)):
        _dev(t, name, torch.int32)
    if k_cache.shape != v_cache.shape or tree_k.shape != tree_v.shape:
        raise ValueError("k/v shapes differ")
    if tree_k.shape[0] != q.shape[0] or parent.shape[0] != q.shape[0]:
        raise ValueError("q, tree_k and parent must have one row per tree node")


def tree_verify_attn_partials(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes,
                              max_prefix_len, max_nodes, workspace, dev_status,
                              softmax_scale=0.0, stream=None, params=None):
    _attn_inputs(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes)
    p = params or make_params(q, k_cache, cu_prefix, cu_nodes, tree_k.shape[1], max_prefix_len,
                              max_nodes, softmax_scale)
    code = load_library().tree_verify_attn_partials(
        ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(tree_k), _ptr(tree_v),
        _ptr(parent), _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _check(code, "tree_verify_attn_partials")


def tree_verify_attn_combine(params: Params, workspace, out, lse, dev_status, stream=None):
    code = load_library().tree_verify_attn_combine(
        ctypes.byref(params), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
        _ptr(dev_status), _stream(stream))
    _check(code, "tree_verify_attn_combine")


def tree_verify_attn_varlen(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes,
                            max_prefix_len, max_nodes, out=None, lse=None, workspace=None,
                            dev_status=None, softmax_scale=0.0, stream=None, params=None):
    """Returns (out [N, Hq, d], lse [N, Hq] float32).  Raises TvaError on a host-side
    error; device-side errors land in ``dev_status`` (allocated and zeroed here when
    not given; check it after synchronising)."""
    _attn_inputs(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes)
    p = params or make_params(q, k_cache, cu_prefix, cu_nodes, tree_k.shape[1], max_prefix_len,
                              max_nodes, softmax_scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(p, q.device)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=q.device)
    code = load_library().tree_verify_attn_varlen(
        ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(tree_k), _ptr(tree_v),
        _ptr(parent), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(dev_status),
        _stream(stream))
    _check(code, "tree_verify_attn_varlen")
    return out, lse


def tree_verify_attn(q, k_cache, v_cache, tree_k, tree_v, parent, out=None, lse=None, stream=None):
    """Single-sequence form: q [m, Hq, d], k_cache/v_cache [P, Hkv, d], tree_k/tree_v
    [m, Hkv, d], parent [m] int32.  Uses the library-owned workspace."""
    _dev(q, "q")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("tree_k", tree_k), ("tree_v", tree_v)):
        _dev(t, name, q.dtype)
    _dev(parent, "parent", torch.int32)
    m, Hq, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((m, Hq), dtype=torch.float32, device=q.device)
    code = load_library().tree_verify_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _ptr(tree_k), _ptr(tree_v),
        _ptr(parent), m, Hq, tree_k.shape[1], d, DTYPES[q.dtype], _ptr(out), _ptr(lse),
        _stream(stream))
    _check(code, "tree_verify_attn")
    return out, lse


def read_device_status(stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(load_library().tva_read_device_status(ctypes.byref(v), _stream(stream)), "tva_read_device_status")
    return int(v.value)


def release():
    load_library().tva_release()


def diag_set_wait_limit(wait_limit_ns: int = 0, force_stall: bool = False):
    """Diagnostics for the device timeout path (tva_diag_set_wait_limit): the main-loop
    wait limit of the tensor-core partials kernel in ns (0 = default 2 s) and, with
    ``force_stall``, a wait that nothing completes.  Call with no arguments to reset."""
    load_library().tva_diag_set_wait_limit(int(wait_limit_ns), 1 if force_stall else 0)


def diag_use_cta_pair(enable: bool = False):
    """Diagnostics (tva_diag_use_cta_pair): select the CTA-pair partials kernel
    (cta_group::2, M = 256) for later calls where it applies; call with no argument to
    return to the default one-SM-per-worker kernel."""
    load_library().tva_diag_use_cta_pair(1 if enable else 0)


def accept_longest_path(cu_nodes, parent, draft_tok, target_argmax, accept_len=None,
                        accept_path=None, next_token=None, dev_status=None, stream=None):
    """Returns (accept_len [B], accept_path [N], next_token [B]) as int32 CUDA tensors."""
    for name, t in (("cu_nodes", cu_nodes), ("parent", parent), ("draft_tok", draft_tok),
                    ("target_argmax", target_argmax)):
        _dev(t, name, torch.int32)
    B = cu_nodes.numel() - 1
    N = parent.numel()
    if target_argmax.numel() != N + B or draft_tok.numel() != N:
        raise ValueError("target_argmax must hold N + B slots and draft_tok N tokens")
    dev = parent.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if accept_path is None:
        accept_path = torch.empty(N, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=dev)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    code = load_library().accept_longest_path(
        B, N, _ptr(cu_nodes), _ptr(parent), _ptr(draft_tok), _ptr(target_argmax), _ptr(accept_len),
        _ptr(accept_path), _ptr(next_token), _ptr(dev_status), _stream(stream))
    _check(code, "accept_longest_path")
    return accept_len, accept_path, next_token


def commit_accepted_kv(cu_nodes, accept_len, accept_path, tree_k, tree_v, dst_row, k_cache, v_cache,
                       max_nodes=None, dev_status=None, stream=None):
    """Copies each sequence's accepted path (root first) of tree_k / tree_v [N, Hkv, d]
    into k_cache / v_cache [rows, Hkv, d] at rows dst_row[b] .. dst_row[b] +
    accept_len[b] - 1, in place.  Returns dev_status (int32 [1], 0 = ok)."""
    for name, t in (("cu_nodes", cu_nodes), ("accept_len", accept_len), ("accept_path", accept_path),
                    ("dst_row", dst_row)):
        _dev(t, name, torch.int32)
    _dev(tree_k, "tree_k")
    for name, t in (("tree_v", tree_v), ("k_cache", k_cache), ("v_cache", v_cache)):
        _dev(t, name, tree_k.dtype)
    if tree_k.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {tree_k.dtype}")
    B = cu_nodes.numel() - 1
    N, Hkv, d = tree_k.shape
    if max_nodes is None:
        max_nodes = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 1
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=tree_k.device)
    code = load_library().commit_accepted_kv(
        B, Hkv, d, DTYPES[tree_k.dtype], N, max(1, int(max_nodes)), k_cache.shape[0], _ptr(cu_nodes),
        _ptr(accept_len), _ptr(accept_path), _ptr(tree_k), _ptr(tree_v), _ptr(dst_row), _ptr(k_cache),
        _ptr(v_cache), _ptr(dev_status), _stream(stream))
    _check(code, "commit_accepted_kv")
    return dev_status


def verify_chain_sampling(cu_draft, p, q, draft_tok, u_accept, u_sample, max_draft=None, accept_len=None,
                          out_token=None, dev_status=None, stream=None):
    """Modified rejection sampling over draft chains.  p [sum(gamma+1), V], q [sum gamma, V]
    float32; draft_tok, u_accept [sum gamma]; u_sample [B]; cu_draft [B+1].
    Returns (accept_len [B], out_token [B]) int32 CUDA tensors."""
    for name, t in (("cu_draft", cu_draft), ("draft_tok", draft_tok)):
        _dev(t, name, torch.int32)
    for name, t in (("p", p), ("q", q), ("u_accept", u_accept), ("u_sample", u_sample)):
        _dev(t, name, torch.float32)
    B = cu_draft.numel() - 1
    V = p.shape[1]
    if q.shape[1] != V and q.numel() > 0:
        raise ValueError("p and q must share the vocabulary")
    if max_draft is None:
        max_draft = int((cu_draft[1:] - cu_draft[:-1]).max().item()) if B > 0 else 0
    dev = p.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if out_token is None:
        out_token = torch.empty(B, dtype=torch.int32, device=dev)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    # with no draft position at all, q / draft_tok / u_accept are never read: any
    # valid address stands in for the empty tensors
    some = lambda t: _ptr(t) if t.numel() > 0 else _ptr(p)  # noqa: E731
    code = load_library().verify_chain_sampling(
        B, V, int(max_draft), p.shape[0], q.shape[0] if q.numel() > 0 else 0, _ptr(cu_draft), _ptr(p), some(q),
        some(draft_tok), some(u_accept), _ptr(u_sample), _ptr(accept_len), _ptr(out_token), _ptr(dev_status),
        _stream(stream))
    _check(code, "verify_chain_sampling")
    return accept_len, out_token


def gdn_tree_verify(cu_nodes, parent, q, k, v, beta, alpha, S0, out=None, max_nodes=None, dev_status=None,
                    stream=None):
    """Gated DeltaNet tree verification.  q, k, v [N, H, d] float32 or bfloat16 (all three
    alike); beta, alpha [N, H] and S0 [B, H, d, d] float32; CUDA tensors.  Returns out
    [N, H, d] in q's dtype."""
    for name, t in (("cu_nodes", cu_nodes), ("parent", parent)):
        _dev(t, name, torch.int32)
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"unsupported dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, q.dtype)
    for name, t in (("beta", beta), ("alpha", alpha), ("S0", S0)):
        _dev(t, name, torch.float32)
    B = cu_nodes.numel() - 1
    N, H, d = q.shape
    if max_nodes is None:
        max_nodes = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 1
    if out is None:
        out = torch.empty_like(v)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=q.device)
    code = load_library().gdn_tree_verify(B, H, d, DTYPES[q.dtype], N, max(1, int(max_nodes)), _ptr(cu_nodes),
                                          _ptr(parent), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha),
                                          _ptr(S0), _ptr(out), _ptr(dev_status), _stream(stream))
    _check(code, "gdn_tree_verify")
    return out


def tree_verify_attn_varlen_noalloc(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes,
                                    max_prefix_len, max_nodes, out=None, lse=None, dev_status=None,
                                    softmax_scale=0.0, stream=None, params=None):
    """tree_verify_attn_varlen without a workspace argument, for callers that may not
    allocate device memory: the library's fixed 32 MiB per-GPU scratch holds the
    partials.  Larger problems raise TvaError (TVA_ERR_WORKSPACE).  Calls share that
    scratch, so calls that overlap on the GPU must be serialised by the caller.
    ``out``, ``lse`` and ``dev_status`` are allocated here only when not given."""
    _attn_inputs(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes)
    lib = load_library()
    fn = lib.tree_verify_attn_varlen_noalloc
    fn.restype = _I
    fn.argtypes = [ctypes.POINTER(Params), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]
    p = params or make_params(q, k_cache, cu_prefix, cu_nodes, tree_k.shape[1], max_prefix_len,
                              max_nodes, softmax_scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=q.device)
    code = fn(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(tree_k), _ptr(tree_v),
              _ptr(parent), _ptr(out), _ptr(lse), _ptr(dev_status), _stream(stream))
    if code != 0:
        detail = lib.tva_last_error().decode()
        raise TvaError(code, "tree_verify_attn_varlen_noalloc" + (f" [{detail}]" if detail else ""))
    return out, lse


# The calls below cost the host about as much as a small call costs the GPU, so their checks
# are few and cheap: one pass over the tensors, pointers as plain integers.

def _c_int(name, value):
    """``value`` for a C int argument: one that does not fit, which ctypes would cut to its low
    bits, and one that is not whole are refused."""
    n = value if type(value) is int else int(value)
    if n != value or not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{name} = {value} is not a 32-bit whole number")
    return n


def _check_all(*named):
    """Each (name, tensor, dtype): contiguous, of that type, on the current device (whose
    stream the kernels run on).  Returns that device's index."""
    here = named[0][1].get_device()
    for name, t, dtype in named:
        if t.get_device() != here or here < 0 or t.dtype is not dtype or not t.is_contiguous():
            _dev(t, name, dtype)
            raise ValueError(f"{name} is on {t.device}, {named[0][0]} on {named[0][1].device}")
    if torch.cuda.current_device() != here:
        raise ValueError(f"the tensors are on cuda:{here}, the current device is cuda:{torch.cuda.current_device()}")
    return here


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device)


def _on_stream(call):
    """With ``stream`` given, runs the call with that stream current: what the call allocates
    then belongs to it, so a status word is zeroed before the kernels write it, and a
    workspace's memory is not handed out again while they still use it."""
    at = list(inspect.signature(call).parameters).index("stream")

    @functools.wraps(call)
    def run(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)

    return run


def _status_word(dev_status, device):
    if dev_status is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    if dev_status.get_device() != device.index or dev_status.dtype is not torch.int32:
        raise ValueError("dev_status must be int32, on the tensors' device")
    return dev_status


def _scale(softmax_scale, d):
    """The logit scale that a call uses (the library's rule)."""
    return softmax_scale if softmax_scale > 0 else d ** -0.5


def _check_plan(p, q, Hkv, rows, cu_prefix, cu_nodes, max_prefix_len, max_nodes, softmax_scale, reported):
    """Refuses a kept plan that is not one of this call: other tensors (a slice of a longer
    cu_prefix starts at the same address, so the batch counts too), another scale than the
    one asked for, or - unless ``reported``, the caller's status word, will tell - lengths
    beyond the plan's bounds."""
    N, Hq, d = q.shape
    if (p.num_q_heads != Hq or p.num_kv_heads != Hkv or p.head_dim != d or p.dtype != DTYPES[q.dtype]
            or p.batch != cu_prefix.shape[0] - 1 or p.node_capacity > N or p.kv_capacity > rows
            or p.cu_prefix != cu_prefix.data_ptr() or p.cu_nodes != cu_nodes.data_ptr()):
        raise ValueError("params do not describe these tensors")
    if softmax_scale != 0:
        mine, plans = _scale(softmax_scale, d), _scale(p.softmax_scale, d)
        if not abs(mine - plans) <= 2.0 ** -22 * plans:  # the plan's is a float32
            raise ValueError(f"params hold another softmax_scale ({plans}) than the call's ({mine})")
    if not reported and ((max_prefix_len is not None and p.max_prefix_len < max_prefix_len)
                         or (max_nodes is not None and p.max_nodes < max_nodes)):
        raise ValueError("params were made for shorter prefixes or smaller trees than the call's")


def _window_attention(name, window, sinks, q, cache, tree_k, tree_v, parent, cu_prefix, cu_nodes, max_prefix_len,
                      max_nodes, out, lse, workspace, dev_status, softmax_scale, params):
    """The checks and the call that the windowed and the 4-bit-cache forms share; ``cache``
    holds (name, tensor, dtype, row shape) of each cache tensor."""
    dt, i32 = q.dtype, torch.int32
    if dt not in DTYPES:
        raise ValueError(f"unsupported dtype {dt}")
    window, sinks = _c_int("window", window), _c_int("sinks", sinks)
    if params is None or max_prefix_len is not None:
        max_prefix_len = _c_int("max_prefix_len", max_prefix_len)
    if params is None or max_nodes is not None:
        max_nodes = _c_int("max_nodes", max_nodes)
    here = _check_all(("q", q, dt), ("tree_k", tree_k, dt), ("tree_v", tree_v, dt), ("parent", parent, i32),
                      ("cu_prefix", cu_prefix, i32), ("cu_nodes", cu_nodes, i32), *(c[:3] for c in cache))
    if q.dim() != 3 or tree_k.dim() != 3 or tree_k.shape != tree_v.shape:
        raise ValueError("q must be [N, Hq, d], tree_k and tree_v [N, Hkv, d]")
    N, Hq, d = q.shape
    Nk, Hkv, dk = tree_k.shape
    if Nk != N or dk != d or parent.shape[0] != N:
        raise ValueError("q, tree_k and parent must have one row per tree node")
    if cu_prefix.dim() != 1 or cu_nodes.shape != cu_prefix.shape:
        raise ValueError("cu_prefix and cu_nodes must hold B + 1 entries each")
    rows = cache[0][1].shape[0]
    for label, t, _, row in cache:
        if t.dim() != 3 or t.shape[0] != rows or t.shape[1] != Hkv or t.shape[2] != row:
            raise ValueError(f"{label} must be [rows, {Hkv}, {row}]")
    p = params
    if p is None:
        p = make_params(q, cache[0][1], cu_prefix, cu_nodes, Hkv, max_prefix_len, max_nodes, softmax_scale)
    else:
        _check_plan(p, q, Hkv, rows, cu_prefix, cu_nodes, max_prefix_len, max_nodes, softmax_scale,
                    dev_status is not None)
    if out is None:
        out = torch.empty_like(q)
    elif out.get_device() != here or out.dtype is not dt or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be like q")
    if lse is None:
        lse = torch.empty((N, Hq), dtype=torch.float32, device=q.device)
    elif (lse.get_device() != here or lse.dtype is not torch.float32 or lse.shape != (N, Hq)
          or not lse.is_contiguous()):
        raise ValueError("lse must be [N, Hq] float32")
    if workspace is None:
        workspace = alloc_workspace(p, q.device)
    elif workspace.get_device() != here or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8, on the tensors' device")
    dev_status = _status_word(dev_status, q.device)
    code = getattr(load_library(), name)(
        ctypes.byref(p), window, sinks, q.data_ptr(), *(c[1].data_ptr() for c in cache), tree_k.data_ptr(),
        tree_v.data_ptr(), parent.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
        dev_status.data_ptr(), _raw_stream(here))
    if code:
        _check(code, name)
    return out, lse


@_on_stream
def tree_verify_attn_window_varlen(q, k_cache, v_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes,
                                   max_prefix_len, max_nodes, window, sinks=0, out=None, lse=None, workspace=None,
                                   dev_status=None, softmax_scale=0.0, stream=None, params=None):
    """tree_verify_attn_varlen under a sliding window: a node at position t (prefix length
    plus proper ancestors) sees the key at position s when ``t - s < window`` or
    ``s < sinks``.  ``window`` >= 1.  Returns (out [N, Hq, d], lse [N, Hq] float32).

    Errors that only the device sees - a bad tree, lengths beyond the bounds, a wait that ran
    out - go to ``dev_status`` (int32 [1], zeroed by the caller) and leave the outputs
    concerned unspecified.  Without it they cannot be seen: pass it, and check it after
    synchronising.

    ``params`` is a plan made by make_params for these tensors and kept; its bounds and its
    scale are then used.  One that does not describe the tensors (their batch included) is
    refused, and so is a ``softmax_scale`` other than its own.  Lengths of the call beyond
    its bounds are refused without ``dev_status``, with it the device reports them.

    While diag_use_cta_pair is on, pass a workspace sized with it off."""
    d = q.shape[-1]
    return _window_attention("tree_verify_attn_window_varlen", window, sinks, q,
                             (("k_cache", k_cache, q.dtype, d), ("v_cache", v_cache, q.dtype, d)), tree_k, tree_v,
                             parent, cu_prefix, cu_nodes, max_prefix_len, max_nodes, out, lse, workspace, dev_status,
                             softmax_scale, params)


@_on_stream
def tree_verify_attn_kv4_varlen(q, kv4_cache, tree_k, tree_v, parent, cu_prefix, cu_nodes, max_prefix_len,
                                max_nodes, window=0, sinks=0, out=None, lse=None, workspace=None, dev_status=None,
                                softmax_scale=0.0, stream=None, params=None):
    """Tree-verification attention whose prefix rows are records of a 4-bit cache; q, tree_k,
    tree_v bf16 or fp16.  ``window`` 0: the whole prefix, else as in
    tree_verify_attn_window_varlen, as are ``dev_status`` (without it a bad tree or length
    cannot be seen) and ``params``.  Returns (out [N, Hq, d], lse [N, Hq] float32)."""
    return _window_attention("tree_verify_attn_kv4_varlen", window, sinks, q,
                             (("kv4_cache", kv4_cache, torch.uint8, kv4_record_bytes(q.shape[-1])),), tree_k, tree_v,
                             parent, cu_prefix, cu_nodes, max_prefix_len, max_nodes, out, lse, workspace, dev_status,
                             softmax_scale, params)


_record_bytes = {}


def kv4_record_bytes(head_dim: int) -> int:
    """Bytes that one row of one KV head takes in a 4-bit cache (K and V together)."""
    n = _record_bytes.get(head_dim)
    if n is None:
        n = int(load_library().tva_kv4_record_bytes(_c_int("head_dim", head_dim)))
        if n == 0:
            raise TvaError(2, "tva_kv4_record_bytes")
        _record_bytes[head_dim] = n
    return n


def alloc_kv4_cache(rows, num_kv_heads, head_dim, device="cuda") -> torch.Tensor:
    """A 4-bit cache [rows, Hkv, record] uint8 of zeros (whose values are all 0)."""
    return torch.zeros((rows, num_kv_heads, kv4_record_bytes(head_dim)), dtype=torch.uint8, device=device)


def _check_records(kv4_cache, num_kv_heads, head_dim):
    record = kv4_record_bytes(head_dim)
    if kv4_cache.dim() != 3 or kv4_cache.shape[1] != num_kv_heads or kv4_cache.shape[2] != record:
        raise ValueError(f"kv4_cache must be [rows, {num_kv_heads}, {record}] uint8")


def _check_rows(k, v):
    if k.dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {k.dtype}")
    if k.dim() != 3 or k.shape != v.shape:
        raise ValueError("k and v must be [rows, Hkv, d], alike")


@_on_stream
def append_kv4(k, v, slot, kv4_cache, dev_status=None, stream=None):
    """Quantises k, v [n, Hkv, d] into rows slot[i] (int32; negative: skipped) of the 4-bit
    cache, in place.  Returns dev_status (int32 [1], 0 = ok)."""
    _check_rows(k, v)
    here = _check_all(("k", k, k.dtype), ("v", v, k.dtype), ("slot", slot, torch.int32),
                      ("kv4_cache", kv4_cache, torch.uint8))
    n, Hkv, d = k.shape
    if slot.shape != (n,):
        raise ValueError("slot must hold one row number per row of k")
    _check_records(kv4_cache, Hkv, d)
    dev_status = _status_word(dev_status, k.device)
    code = load_library().append_kv4(n, Hkv, d, DTYPES[k.dtype], kv4_cache.shape[0], k.data_ptr(), v.data_ptr(),
                                     slot.data_ptr(), kv4_cache.data_ptr(), dev_status.data_ptr(),
                                     _raw_stream(here))
    if code:
        _check(code, "append_kv4")
    return dev_status


@_on_stream
def read_kv4(kv4_cache, head_dim, slot=None, dtype=torch.bfloat16, k=None, v=None, dev_status=None, stream=None):
    """(k, v) [n, Hkv, head_dim] of ``dtype``: the values that rows slot[i] (int32; negative:
    zeros) of the 4-bit cache stand for, or all rows in order when ``slot`` is None.  A slot
    beyond the cache reads as zeros too and is reported in ``dev_status`` (int32 [1], zeroed
    by the caller); without it that cannot be seen."""
    if dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    here = _check_all(("kv4_cache", kv4_cache, torch.uint8))
    _check_records(kv4_cache, kv4_cache.shape[1] if kv4_cache.dim() == 3 else 0, head_dim)
    rows, Hkv, _ = kv4_cache.shape
    n = rows
    if slot is not None:
        _check_all(("slot", slot, torch.int32))
        if slot.dim() != 1:
            raise ValueError("slot must be one-dimensional")
        n = slot.shape[0]
    shape = (n, Hkv, int(head_dim))
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=kv4_cache.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=kv4_cache.device)
    _check_all(("k", k, dtype), ("v", v, dtype))
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k and v must be {list(shape)}")
    dev_status = _status_word(dev_status, kv4_cache.device)
    code = load_library().read_kv4(n, Hkv, shape[2], DTYPES[dtype], rows, kv4_cache.data_ptr(),
                                   None if slot is None else slot.data_ptr(), k.data_ptr(), v.data_ptr(),
                                   dev_status.data_ptr(), _raw_stream(here))
    if code:
        _check(code, "read_kv4")
    return k, v


@_on_stream
def commit_accepted_kv4(cu_nodes, accept_len, accept_path, tree_k, tree_v, dst_row, kv4_cache, max_nodes=None,
                        dev_status=None, stream=None):
    """commit_accepted_kv into a 4-bit cache [rows, Hkv, record], in place.  Returns
    dev_status (int32 [1], 0 = ok)."""
    _check_rows(tree_k, tree_v)
    if max_nodes is not None:
        max_nodes = _c_int("max_nodes", max_nodes)
    dt, i32 = tree_k.dtype, torch.int32
    here = _check_all(("cu_nodes", cu_nodes, i32), ("accept_len", accept_len, i32), ("accept_path", accept_path, i32),
                      ("dst_row", dst_row, i32), ("tree_k", tree_k, dt), ("tree_v", tree_v, dt),
                      ("kv4_cache", kv4_cache, torch.uint8))
    B = cu_nodes.shape[0] - 1
    N, Hkv, d = tree_k.shape
    if accept_len.shape[0] != B or dst_row.shape[0] != B or accept_path.shape[0] != N:
        raise ValueError("accept_len and dst_row must hold B entries and accept_path one per node")
    _check_records(kv4_cache, Hkv, d)
    if max_nodes is None:
        max_nodes = int((cu_nodes[1:] - cu_nodes[:-1]).max().item()) if B > 0 else 1
    dev_status = _status_word(dev_status, tree_k.device)
    code = load_library().commit_accepted_kv4(
        B, Hkv, d, DTYPES[dt], N, max(1, max_nodes), kv4_cache.shape[0], cu_nodes.data_ptr(),
        accept_len.data_ptr(), accept_path.data_ptr(), tree_k.data_ptr(), tree_v.data_ptr(), dst_row.data_ptr(),
        kv4_cache.data_ptr(), dev_status.data_ptr(), _raw_stream(here))
    if code:
        _check(code, "commit_accepted_kv4")
    return dev_status
