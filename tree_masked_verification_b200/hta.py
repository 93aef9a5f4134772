"""ctypes binding of liblongspec_hta.so (Hybrid Tree Attention on B200).

Argument marshalling only: every step of the verification attention runs in
the library's CUDA kernels.  Tensors are torch tensors on the current CUDA
device; the library launches on torch's current stream unless a stream is
given (what a call then allocates itself is memory of that stream; what it
is given has to be ready there).  The library must have been built (``tree_masked_verification_b200.build``):
there is no fallback of any kind, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

# The in-tree build; LONGSPEC_HTA_LIB names another build of the same
# library instead (a build with other tuning knobs, for A/B timing).
_LIB_PATH = os.environ.get("LONGSPEC_HTA_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "liblongspec_hta.so")
_lock = threading.Lock()
_lib = None

OK = 0
ERR_INVALID_DIMS = -1
ERR_NULL_POINTER = -2
ERR_MISALIGNED = -3
ERR_T_TOO_LARGE = -4
ERR_UNSUPPORTED_D = -5
ERR_WORKSPACE_TOO_SMALL = -6
ERR_CUDA = -7
ERR_UNSUPPORTED_DEVICE = -8
ERR_INVALID_OPTION = -9
ERR_BAD_PARENT = -16
ERR_PREFIX_LEN_RANGE = -17
ERR_PIPELINE_TIMEOUT = -18
ERR_INTERNAL = -19
ERR_BAD_BLOCK = -20
ERR_BAD_PATH = -21
ERR_BAD_RANGES = -22

PREFIX_TCGEN05 = 0
PREFIX_SIMT = 1
T_MAX = 256

EXPORTED = [
    "longspec_hta_abi_version", "longspec_hta_build_info", "longspec_hta_strerror", "longspec_hta_default_splits",
    "longspec_hta_chunking",
    "longspec_hta_workspace_bytes", "longspec_hta_workspace_init", "longspec_hta_verify",
    "longspec_hta_verify_ex", "longspec_hta_host_arena_bytes", "longspec_hta_verify_host",
    "longspec_hta_tree_mask", "longspec_hta_tree_partial", "longspec_hta_prefix_partial",
    "longspec_hta_get_status", "longspec_hta_verify_noalloc", "longspec_hta_noalloc_chunking",
    "longspec_hta_selftest_wait_timeout", "longspec_hta_prefix_attention",
    "longspec_hta_verify_paged", "longspec_hta_prefix_attention_paged",
    "longspec_hta_accept_workspace_bytes", "longspec_hta_accept_greedy",
    "longspec_hta_commit", "longspec_hta_commit_paged", "longspec_hta_window_verify",
    "longspec_hta_window_workspace_bytes",
    "longspec_hta_qk_norm_rope", "longspec_hta_append_paged", "longspec_hta_chunk_workspace_bytes",
    "longspec_hta_chunk_attention_paged", "longspec_hta_q8_workspace_bytes", "longspec_hta_verify_paged_q8",
    "longspec_hta_prefix_attention_paged_q8", "longspec_hta_commit_paged_q8",
]


class HtaError(RuntimeError):
    def __init__(self, code: int):
        msg = load().longspec_hta_strerror(code).decode()
        super().__init__(f"longspec_hta error {code}: {msg}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("T", ctypes.c_int), ("L_cap", ctypes.c_int),
                ("scale", ctypes.c_float)]


class Options(ctypes.Structure):
    _fields_ = [("num_splits", ctypes.c_int), ("prefix_kernel", ctypes.c_int),
                ("prefix_begin", ctypes.c_void_p), ("prefix_end", ctypes.c_void_p)]


class PagedKV(ctypes.Structure):
    """longspec_hta_paged_kv: caches [num_blocks][Hkv][block_size][D] bf16,
    block_table [B][max_blocks] int32 (device pointers)."""
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("num_blocks", ctypes.c_int),
                ("block_size", ctypes.c_int), ("max_blocks", ctypes.c_int)]


class Cache(ctypes.Structure):
    """longspec_hta_cache: a paged cache, bf16 or (with scales) e4m3."""
    _fields_ = PagedKV._fields_ + [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class Rope(ctypes.Structure):
    """longspec_hta_rope: frequencies and norm weights of query and key heads."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load the library (once).  Raises if it was not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with "
                    "`python -m tree_masked_verification_b200.build` (no fallback exists)")
            lib = ctypes.CDLL(_LIB_PATH)
            vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            pd = ctypes.POINTER(Dims)
            lib.longspec_hta_abi_version.restype = ci
            lib.longspec_hta_build_info.restype = ctypes.c_char_p
            lib.longspec_hta_strerror.argtypes = [ci]
            lib.longspec_hta_strerror.restype = ctypes.c_char_p
            lib.longspec_hta_default_splits.argtypes = [pd]
            lib.longspec_hta_workspace_bytes.argtypes = [pd, ci]
            lib.longspec_hta_workspace_bytes.restype = sz
            lib.longspec_hta_workspace_init.argtypes = [vp, sz, vp]
            lib.longspec_hta_verify.argtypes = [pd] + [vp] * 9 + [vp, sz, vp]
            lib.longspec_hta_verify_ex.argtypes = [pd] + [vp] * 9 + [vp, sz, ctypes.POINTER(Options), vp]
            lib.longspec_hta_prefix_attention.argtypes = [pd] + [vp] * 6 + [vp, sz, ctypes.POINTER(Options), vp]
            pk = ctypes.POINTER(PagedKV)
            lib.longspec_hta_verify_paged.argtypes = [pd, vp, pk] + [vp] * 6 + [vp, sz, ctypes.POINTER(Options), vp]
            lib.longspec_hta_prefix_attention_paged.argtypes = [pd, vp, pk] + [vp] * 3 + [vp, sz, ctypes.POINTER(Options), vp]
            lib.longspec_hta_host_arena_bytes.argtypes = [pd]
            lib.longspec_hta_host_arena_bytes.restype = sz
            lib.longspec_hta_verify_host.argtypes = [pd] + [vp] * 9 + [vp, sz, vp]
            lib.longspec_hta_tree_mask.argtypes = [vp, ci, ci, vp, vp, sz, vp]
            lib.longspec_hta_tree_partial.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            lib.longspec_hta_prefix_partial.argtypes = [pd, vp, vp, vp, vp, vp, vp, ci, ci,
                                                        ctypes.POINTER(ci), vp, sz, vp]
            lib.longspec_hta_get_status.argtypes = [vp, vp]
            lib.longspec_hta_selftest_wait_timeout.argtypes = [vp, vp]
            lib.longspec_hta_chunking.argtypes = [pd, ci, ctypes.POINTER(ci), ctypes.POINTER(ci)]
            lib.longspec_hta_noalloc_chunking.argtypes = [pd, ci, ctypes.POINTER(ci), ctypes.POINTER(ci)]
            lib.longspec_hta_accept_workspace_bytes.argtypes = [ci, ci, ci]
            lib.longspec_hta_accept_workspace_bytes.restype = sz
            lib.longspec_hta_accept_greedy.argtypes = [ci, ci, ci] + [vp] * 6 + [vp, sz, vp]
            lib.longspec_hta_commit.argtypes = [pd] + [vp] * 7 + [vp, sz, vp]
            lib.longspec_hta_window_verify.argtypes = [pd] + [vp] * 9 + [vp, sz, vp]
            lib.longspec_hta_window_workspace_bytes.argtypes = [pd]
            lib.longspec_hta_window_workspace_bytes.restype = sz
            lib.longspec_hta_commit_paged.argtypes = [pd, pk] + [vp] * 5 + [vp, sz, vp]
            pr, pc = ctypes.POINTER(Rope), ctypes.POINTER(Cache)
            # (longspec_hta_heads go over as packed bytes)
            lib.longspec_hta_qk_norm_rope.argtypes = [ci] * 5 + [vp, vp, vp, pr, vp, vp, vp]
            lib.longspec_hta_append_paged.argtypes = [pd, vp, vp, vp, pr, pc, vp, vp, vp, vp, sz, vp]
            lib.longspec_hta_chunk_workspace_bytes.argtypes = [pd]
            lib.longspec_hta_chunk_workspace_bytes.restype = sz
            lib.longspec_hta_chunk_attention_paged.argtypes = [pd, vp, pc, vp, vp, ci] + [vp] * 3 + [sz, vp]
            lib.longspec_hta_q8_workspace_bytes.argtypes = [pd]
            lib.longspec_hta_q8_workspace_bytes.restype = sz
            lib.longspec_hta_verify_paged_q8.argtypes = [pd, vp, pc] + [vp] * 7 + [sz, vp]
            lib.longspec_hta_prefix_attention_paged_q8.argtypes = [pd, vp, pc] + [vp] * 4 + [sz, vp]
            lib.longspec_hta_commit_paged_q8.argtypes = [pd, pc] + [vp] * 6 + [sz, vp]
            _lib = lib
    return _lib


def _check(rc: int):
    if rc != OK:
        raise HtaError(rc)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _new(stream, make, *args, **kwargs):
    """make(...): a tensor that the call allocates itself.  With a stream of
    the caller's it is memory of that stream: filled before the kernels that
    read it, and not handed out again before they have run.  What the call
    returns may be used, once it is waited for, on the stream that is current
    now."""
    if stream is None:
        return make(*args, **kwargs)
    side = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    here = torch.cuda.current_stream()
    with torch.cuda.stream(side):
        t = make(*args, **kwargs)
    t.record_stream(here)
    return t


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def dims_of(q: torch.Tensor, k_prefix: torch.Tensor, scale: float = 0.0) -> Dims:
    B, Hq, T, D = q.shape
    return Dims(B, Hq, k_prefix.shape[1], D, T, k_prefix.shape[2], float(scale))


def _need(t: torch.Tensor, name: str, dtype, device=None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def default_splits(dims: Dims) -> int:
    rc = load().longspec_hta_default_splits(ctypes.byref(dims))
    if rc < 0:
        raise HtaError(rc)
    return rc


def chunking(dims: Dims, num_splits: int = 0):
    """(S, chunk_keys) the library uses for a requested split count."""
    S, C = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().longspec_hta_chunking(ctypes.byref(dims), int(num_splits), ctypes.byref(S),
                                        ctypes.byref(C)))
    return S.value, C.value


def noalloc_chunking(dims: Dims, num_sms: int):
    """(S, chunk_keys) longspec_hta_verify_noalloc uses on a GPU with
    num_sms SMs (host only)."""
    S, C = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().longspec_hta_noalloc_chunking(ctypes.byref(dims), int(num_sms), ctypes.byref(S),
                                                ctypes.byref(C)))
    return S.value, C.value


def workspace_bytes(dims: Dims, num_splits: int = 0) -> int:
    n = load().longspec_hta_workspace_bytes(ctypes.byref(dims), int(num_splits))
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return n


def new_workspace(dims: Dims, num_splits: int = 0, device=None) -> torch.Tensor:
    """A zeroed device workspace for verify (status word cleared)."""
    return torch.zeros(workspace_bytes(dims, num_splits), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def verify(q, k_prefix, v_prefix, prefix_len, k_tree, v_tree, parent, *, out=None,
           lse=None, workspace=None, scale: float = 0.0, num_splits: int = 0,
           prefix_kernel: int = PREFIX_TCGEN05, prefix_events=None, stream=None):
    """Hybrid Tree Attention of one layer.  Returns (out bf16, lse fp32)."""
    dev = q.device
    for t, n in ((q, "q"), (k_prefix, "k_prefix"), (v_prefix, "v_prefix"),
                 (k_tree, "k_tree"), (v_tree, "v_tree")):
        _need(t, n, torch.bfloat16, dev)
    _need(prefix_len, "prefix_len", torch.int32, dev)
    _need(parent, "parent", torch.int32, dev)
    dims = dims_of(q, k_prefix, scale)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    if lse is None:
        lse = _new(stream, torch.empty, q.shape[:3], dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _new(stream, new_workspace, dims, num_splits, dev)
    opts = Options(int(num_splits), int(prefix_kernel),
                   prefix_events[0].cuda_event if prefix_events else None,
                   prefix_events[1].cuda_event if prefix_events else None)
    rc = load().longspec_hta_verify_ex(
        ctypes.byref(dims), _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(prefix_len),
        _ptr(k_tree), _ptr(v_tree), _ptr(parent), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(opts), _stream(stream))
    _check(rc)
    return out, lse


def prefix_attention(q, k_prefix, v_prefix, prefix_len, *, out=None, lse=None, workspace=None,
                     scale: float = 0.0, num_splits: int = 0, prefix_kernel: int = PREFIX_TCGEN05,
                     prefix_events=None, stream=None):
    """Attention of q's rows to the prefix alone (no tree keys, no mask):
    the draft model's cross-attention into the target's KV cache.  q is
    [B][Hq][T][D] with T query tokens per head.  Returns (out bf16, lse fp32);
    rows of a sequence with L_b = 0 get out 0 and lse -inf."""
    dev = q.device
    for t, n in ((q, "q"), (k_prefix, "k_prefix"), (v_prefix, "v_prefix")):
        _need(t, n, torch.bfloat16, dev)
    _need(prefix_len, "prefix_len", torch.int32, dev)
    dims = dims_of(q, k_prefix, scale)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    if lse is None:
        lse = _new(stream, torch.empty, q.shape[:3], dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _new(stream, new_workspace, dims, num_splits, dev)
    opts = Options(int(num_splits), int(prefix_kernel),
                   prefix_events[0].cuda_event if prefix_events else None,
                   prefix_events[1].cuda_event if prefix_events else None)
    rc = load().longspec_hta_prefix_attention(
        ctypes.byref(dims), _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(prefix_len),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        ctypes.byref(opts), _stream(stream))
    _check(rc)
    return out, lse


def _paged(k_cache, v_cache, block_table, dev):
    _need(k_cache, "k_cache", torch.bfloat16, dev)
    _need(v_cache, "v_cache", torch.bfloat16, dev)
    _need(block_table, "block_table", torch.int32, dev)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or block_table.dim() != 2:
        raise ValueError("k/v_cache must be [num_blocks][Hkv][block_size][D], block_table [B][max_blocks]")
    return PagedKV(_ptr(k_cache), _ptr(v_cache), _ptr(block_table), int(k_cache.shape[0]),
                   int(k_cache.shape[2]), int(block_table.shape[1]))


def _paged_dims(q, k_cache, L_cap, scale):
    B, Hq, T, D = q.shape
    return Dims(B, Hq, int(k_cache.shape[1]), D, T, int(L_cap), float(scale))


def verify_paged(q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, parent, *, L_cap,
                 out=None, lse=None, workspace=None, scale: float = 0.0, num_splits: int = 0,
                 prefix_events=None, stream=None, k_scale=None, v_scale=None):
    """verify() with the prefix K/V in a paged cache: k/v_cache
    [num_blocks][Hkv][block_size][D], block_table [B][max_blocks] (block ids
    of each sequence in key order), L_cap the longest prefix allowed.

    With k_scale and v_scale (uint8 [num_blocks][Hkv][block_size]) the caches
    hold e4m3 codes (see append_paged); the workspace is then one of
    new_q8_workspace(), and num_splits and prefix_events do not apply."""
    dev = q.device
    if k_scale is not None or v_scale is not None:
        return _attention_q8(q, k_cache, v_cache, block_table, prefix_len, (k_tree, v_tree, parent), L_cap, out, lse,
                             workspace, scale, num_splits, prefix_events, stream, k_scale, v_scale)
    for t, n in ((q, "q"), (k_tree, "k_tree"), (v_tree, "v_tree")):
        _need(t, n, torch.bfloat16, dev)
    _need(prefix_len, "prefix_len", torch.int32, dev)
    _need(parent, "parent", torch.int32, dev)
    kv = _paged(k_cache, v_cache, block_table, dev)
    dims = _paged_dims(q, k_cache, L_cap, scale)
    out = _new(stream, torch.empty_like, q) if out is None else out
    lse = _new(stream, torch.empty, q.shape[:3], dtype=torch.float32, device=dev) if lse is None else lse
    workspace = _new(stream, new_workspace, dims, num_splits, dev) if workspace is None else workspace
    opts = Options(int(num_splits), PREFIX_TCGEN05,
                   prefix_events[0].cuda_event if prefix_events else None,
                   prefix_events[1].cuda_event if prefix_events else None)
    rc = load().longspec_hta_verify_paged(
        ctypes.byref(dims), _ptr(q), ctypes.byref(kv), _ptr(prefix_len), _ptr(k_tree), _ptr(v_tree),
        _ptr(parent), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(opts), _stream(stream))
    _check(rc)
    return out, lse


def prefix_attention_paged(q, k_cache, v_cache, block_table, prefix_len, *, L_cap, out=None,
                           lse=None, workspace=None, scale: float = 0.0, num_splits: int = 0,
                           prefix_events=None, stream=None, k_scale=None, v_scale=None):
    """prefix_attention() with the prefix K/V in a paged cache, in bf16 or,
    with k_scale and v_scale, in e4m3 (as in verify_paged)."""
    dev = q.device
    if k_scale is not None or v_scale is not None:
        return _attention_q8(q, k_cache, v_cache, block_table, prefix_len, None, L_cap, out, lse, workspace, scale,
                             num_splits, prefix_events, stream, k_scale, v_scale)
    _need(q, "q", torch.bfloat16, dev)
    _need(prefix_len, "prefix_len", torch.int32, dev)
    kv = _paged(k_cache, v_cache, block_table, dev)
    dims = _paged_dims(q, k_cache, L_cap, scale)
    out = _new(stream, torch.empty_like, q) if out is None else out
    lse = _new(stream, torch.empty, q.shape[:3], dtype=torch.float32, device=dev) if lse is None else lse
    workspace = _new(stream, new_workspace, dims, num_splits, dev) if workspace is None else workspace
    opts = Options(int(num_splits), PREFIX_TCGEN05,
                   prefix_events[0].cuda_event if prefix_events else None,
                   prefix_events[1].cuda_event if prefix_events else None)
    rc = load().longspec_hta_prefix_attention_paged(
        ctypes.byref(dims), _ptr(q), ctypes.byref(kv), _ptr(prefix_len), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel() * workspace.element_size(), ctypes.byref(opts),
        _stream(stream))
    _check(rc)
    return out, lse


def host_arena_bytes(dims: Dims) -> int:
    n = load().longspec_hta_host_arena_bytes(ctypes.byref(dims))
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return n


def verify_host(q, k_prefix, v_prefix, prefix_len, k_tree, v_tree, parent, out, lse,
                arena, *, scale: float = 0.0, stream=None):
    """End-to-end call on host tensors (pinned for asynchronous copies): the
    library copies inputs into the device `arena`, runs, and copies out/lse
    back on `stream`.  Synchronise the stream before reading out/lse."""
    for t, n in ((q, "q"), (k_prefix, "k_prefix"), (v_prefix, "v_prefix"),
                 (k_tree, "k_tree"), (v_tree, "v_tree"), (out, "out")):
        _need(t, n, torch.bfloat16, torch.device("cpu"))
    _need(prefix_len, "prefix_len", torch.int32, torch.device("cpu"))
    _need(parent, "parent", torch.int32, torch.device("cpu"))
    _need(lse, "lse", torch.float32, torch.device("cpu"))
    dims = dims_of(q, k_prefix, scale)
    rc = load().longspec_hta_verify_host(
        ctypes.byref(dims), _ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(prefix_len),
        _ptr(k_tree), _ptr(v_tree), _ptr(parent), _ptr(out), _ptr(lse), _ptr(arena),
        arena.numel() * arena.element_size(), _stream(stream))
    _check(rc)


def tree_mask(parent: torch.Tensor, workspace=None, stream=None) -> torch.Tensor:
    """Ancestor-or-self bits uint32-as-int32 [B][T][ceil(T/32)] (debug export)."""
    _need(parent, "parent", torch.int32)
    B, T = parent.shape
    W = (T + 31) // 32
    bits = _new(stream, torch.empty, B, T, W, dtype=torch.int32, device=parent.device)
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=parent.device)
    _check(load().longspec_hta_tree_mask(_ptr(parent), B, T, _ptr(bits), _ptr(workspace),
                                         workspace.numel(), _stream(stream)))
    return bits


def tree_partial(q, k_tree, v_tree, parent, *, scale: float = 0.0, workspace=None, stream=None):
    """Tree-only partial (debug export): (o_tree fp32 [B][Hq][T][D], lse_tree fp32)."""
    B, Hq, T, D = q.shape
    dims = Dims(B, Hq, k_tree.shape[1], D, T, 0, float(scale))
    o = _new(stream, torch.empty, B, Hq, T, D, dtype=torch.float32, device=q.device)
    l = _new(stream, torch.empty, B, Hq, T, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=q.device)
    _check(load().longspec_hta_tree_partial(ctypes.byref(dims), _ptr(q), _ptr(k_tree),
                                            _ptr(v_tree), _ptr(parent), _ptr(o), _ptr(l),
                                            _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, l


def prefix_partial(q, k_prefix, v_prefix, prefix_len, *, scale: float = 0.0,
                   num_splits: int = 0, prefix_kernel: int = PREFIX_TCGEN05,
                   workspace=None, stream=None):
    """Split-KV prefix partials (debug export):
    (o_part fp32 [B][Hq][T][S][D], lse_part fp32 [B][Hq][T][S], chunk keys)."""
    dims = dims_of(q, k_prefix, scale)
    lib = load()
    # the default call's split count, passed on explicitly so that every
    # prefix kernel cuts the keys the same way
    S, chunk_keys = chunking(dims, num_splits)
    S_out = ctypes.c_int(0)
    B, Hq, T, D = q.shape
    o = _new(stream, torch.empty, B, Hq, T, S, D, dtype=torch.float32, device=q.device)
    l = _new(stream, torch.empty, B, Hq, T, S, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=q.device)
    _check(lib.longspec_hta_prefix_partial(ctypes.byref(dims), _ptr(q), _ptr(k_prefix),
                                           _ptr(v_prefix), _ptr(prefix_len), _ptr(o), _ptr(l),
                                           int(S), int(prefix_kernel), ctypes.byref(S_out),
                                           _ptr(workspace), workspace.numel(), _stream(stream)))
    if S_out.value != S:
        raise RuntimeError(f"split count mismatch: library {S_out.value}, binding {S}")
    return o, l, chunk_keys


def accept_workspace_bytes(B: int, T: int, V: int) -> int:
    return int(load().longspec_hta_accept_workspace_bytes(int(B), int(T), int(V)))


def new_accept_workspace(B: int, T: int, V: int, device=None) -> torch.Tensor:
    n = accept_workspace_bytes(B, T, V)
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def accept_greedy(logits, draft_tokens, parent, *, accept_len=None, path=None, bonus=None,
                  workspace=None, stream=None):
    """Greedy (temperature 0) acceptance of the draft tree.

    logits bf16 [B][T+1][V] (row 0: the prefix end, row 1+i: after node i),
    draft_tokens and parent int32 [B][T].  Returns (accept_len int32 [B],
    path int32 [B][T] padded with -1, bonus int32 [B])."""
    _need(logits, "logits", torch.bfloat16)
    dev = logits.device
    _need(draft_tokens, "draft_tokens", torch.int32, dev)
    _need(parent, "parent", torch.int32, dev)
    B, T1, V = logits.shape
    T = T1 - 1
    if tuple(draft_tokens.shape) != (B, T) or tuple(parent.shape) != (B, T):
        raise ValueError(f"draft_tokens/parent must be [{B}][{T}]")
    if accept_len is None:
        accept_len = _new(stream, torch.empty, B, dtype=torch.int32, device=dev)
    if path is None:
        path = _new(stream, torch.empty, B, T, dtype=torch.int32, device=dev)
    if bonus is None:
        bonus = _new(stream, torch.empty, B, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _new(stream, new_accept_workspace, B, T, V, dev)
    _check(load().longspec_hta_accept_greedy(
        B, T, V, _ptr(logits), _ptr(draft_tokens), _ptr(parent), _ptr(accept_len), _ptr(path),
        _ptr(bonus), _ptr(workspace), workspace.numel(), _stream(stream)))
    return accept_len, path, bonus


def new_window_workspace(dims: Dims, device=None) -> torch.Tensor:
    n = int(load().longspec_hta_window_workspace_bytes(ctypes.byref(dims)))
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def window_verify(q, k_ring, v_ring, prefix_len, k_tree, v_tree, parent, *, out=None, lse=None,
                  workspace=None, scale: float = 0.0, stream=None):
    """Sliding-window tree attention (the draft model's self-attention): the
    ring k/v_ring [B][Hkv][W][D] holds context position p at slot p mod W;
    a node at depth d sees its root path and positions [L_b + d - W, L_b)."""
    _need(q, "q", torch.bfloat16)
    dev = q.device
    for t, n in ((k_ring, "k_ring"), (v_ring, "v_ring"), (k_tree, "k_tree"), (v_tree, "v_tree")):
        _need(t, n, torch.bfloat16, dev)
    _need(prefix_len, "prefix_len", torch.int32, dev)
    _need(parent, "parent", torch.int32, dev)
    dims = dims_of(q, k_ring, scale)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    if lse is None:
        lse = _new(stream, torch.empty, q.shape[:3], dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _new(stream, new_window_workspace, dims, dev)
    _check(load().longspec_hta_window_verify(
        ctypes.byref(dims), _ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(prefix_len), _ptr(k_tree),
        _ptr(v_tree), _ptr(parent), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return out, lse


def _commit_dims(k_tree, L_cap):
    B, Hkv, T, D = k_tree.shape
    return Dims(B, Hkv, Hkv, D, T, int(L_cap), 0.0)


def commit(k_prefix, v_prefix, prefix_len, k_tree, v_tree, accept_len, path, *, workspace=None,
           stream=None):
    """Append the accepted path's tree K/V rows to the contiguous cache
    [B][Hkv][L_cap][D] after each prefix and advance prefix_len in place."""
    for t, n in ((k_prefix, "k_prefix"), (v_prefix, "v_prefix"), (k_tree, "k_tree"), (v_tree, "v_tree")):
        _need(t, n, torch.bfloat16, k_tree.device)
    for t, n in ((prefix_len, "prefix_len"), (accept_len, "accept_len"), (path, "path")):
        _need(t, n, torch.int32, k_tree.device)
    dims = _commit_dims(k_tree, k_prefix.shape[2])
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=k_tree.device)
    _check(load().longspec_hta_commit(ctypes.byref(dims), _ptr(k_prefix), _ptr(v_prefix),
                                      _ptr(prefix_len), _ptr(k_tree), _ptr(v_tree),
                                      _ptr(accept_len), _ptr(path), _ptr(workspace),
                                      workspace.numel(), _stream(stream)))


def commit_paged(k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, accept_len, path, *,
                 L_cap, workspace=None, stream=None, k_scale=None, v_scale=None):
    """commit() into a paged cache [num_blocks][Hkv][block_size][D], in bf16
    or, with k_scale and v_scale, in e4m3 (the rows are then stored as
    append_paged stores them)."""
    if k_scale is not None or v_scale is not None:
        dev = k_tree.get_device()
        ptrs = [_flat(t, n, _BF16, dev) for t, n in ((k_tree, "k_tree"), (v_tree, "v_tree"))]
        ptrs += [_flat(t, n, _I32, dev) for t, n in ((accept_len, "accept_len"), (path, "path"))]
        pre = _flat(prefix_len, "prefix_len", _I32, dev)
        cache = _cache(k_cache, v_cache, block_table, k_scale, v_scale, dev)
        dims = _commit_dims(k_tree, L_cap)
        _tree_shapes(dims, k_cache, prefix_len, block_table, k_tree, v_tree, path)
        if accept_len.shape != (dims.B,):
            raise ValueError(f"accept_len must be [{dims.B}]")
        st = _stream_on(dev, stream)
        if workspace is None:
            workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=k_tree.device)
        _check(load().longspec_hta_commit_paged_q8(
            dims, cache, pre, *ptrs, _flat(workspace, "workspace", torch.uint8, dev), workspace.nbytes, st))
        return
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_tree, "k_tree"), (v_tree, "v_tree")):
        _need(t, n, torch.bfloat16, k_tree.device)
    for t, n in ((block_table, "block_table"), (prefix_len, "prefix_len"), (accept_len, "accept_len"),
                 (path, "path")):
        _need(t, n, torch.int32, k_tree.device)
    dims = _commit_dims(k_tree, L_cap)
    kv = _paged(k_cache, v_cache, block_table, k_tree.device)
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=k_tree.device)
    _check(load().longspec_hta_commit_paged(ctypes.byref(dims), ctypes.byref(kv), _ptr(prefix_len),
                                            _ptr(k_tree), _ptr(v_tree), _ptr(accept_len), _ptr(path),
                                            _ptr(workspace), workspace.numel(), _stream(stream)))


# ---- new tokens: norm, rotation, append, chunk attention; the e4m3 cache ----

# These calls are short on the device, so the binding keeps its own time
# short: device indices are compared as ints, row descriptors are packed bytes,
# the current stream is read as the raw handle.

_BF16, _I32 = torch.bfloat16, torch.int32
_heads_struct = struct.Struct("4q").pack          # longspec_hta_heads
_contiguous = torch.contiguous_format


def _stream_on(dev: int, stream) -> int:
    """The stream to launch on; the tensors must be on the current device."""
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return _stream(stream)


def _like(t, stream):
    """A contiguous tensor of t's shape for a call's result."""
    if stream is None:
        return torch.empty_like(t, memory_format=_contiguous)
    return _new(stream, torch.empty_like, t, memory_format=_contiguous)


def _flat(t, name, dtype, dev: int):
    """A contiguous tensor's pointer."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _result(t, name, shape, dtype, dev: int):
    _flat(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _cache(k_cache, v_cache, block_table, k_scale, v_scale, dev: int) -> Cache:
    shape = k_cache.shape
    if len(shape) != 4 or shape != v_cache.shape or block_table.dim() != 2:
        raise ValueError("k/v_cache must be [num_blocks][Hkv][block_size][D], block_table [B][max_blocks]")
    dtype, ks, vs = _BF16, None, None
    if k_scale is not None or v_scale is not None:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache has both k_scale and v_scale")
        dtype = torch.float8_e4m3fn
        ks, vs = _flat(k_scale, "k_scale", torch.uint8, dev), _flat(v_scale, "v_scale", torch.uint8, dev)
        if k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
            raise ValueError("k_scale and v_scale must be [num_blocks][Hkv][block_size]")
    return Cache(_flat(k_cache, "k_cache", dtype, dev), _flat(v_cache, "v_cache", dtype, dev),
                 _flat(block_table, "block_table", _I32, dev), shape[0], shape[2], block_table.shape[1], ks, vs)


def _tree_shapes(dims, k_cache, prefix_len, block_table, k_tree=None, v_tree=None, nodes=None):
    if k_cache.shape[1] != dims.Hkv or k_cache.shape[3] != dims.D:
        raise ValueError(f"the cache holds {k_cache.shape[1]} heads of {k_cache.shape[3]}")
    if prefix_len.shape != (dims.B,) or block_table.shape[0] != dims.B:
        raise ValueError(f"prefix_len must be [{dims.B}], block_table [{dims.B}][max_blocks]")
    if k_tree is not None and (k_tree.shape != (dims.B, dims.Hkv, dims.T, dims.D) or v_tree.shape != k_tree.shape
                               or nodes.shape != (dims.B, dims.T)):
        raise ValueError(f"k/v_tree must be [{dims.B}][{dims.Hkv}][{dims.T}][{dims.D}] and the node array "
                         f"[{dims.B}][{dims.T}]")


def _heads(t, name, dev: int, b, n, h):
    """longspec_hta_heads of a bf16 tensor whose rows are D contiguous values;
    b, n, h: its axes (batch, token, head), b -1 for none."""
    if t.dtype != _BF16:
        raise TypeError(f"{name}: expected {_BF16}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    sb, sn, sh = 0 if b < 0 else st[b], st[n], st[h]
    if (sb | sn | sh) & 7:           # (the stride of an axis of one means nothing)
        sb, sn, sh = (x if t.shape[i] > 1 else 0 for x, i in ((sb, b), (sn, n), (sh, h)))
    return _heads_struct(t.data_ptr(), sb, sn, sh)


def _rope(inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, D, dev: int) -> Rope:
    f = _flat(inv_freq, "inv_freq", torch.float32, dev)
    if inv_freq.dim() != 1 or not 1 <= inv_freq.shape[0] <= D // 2:
        raise ValueError(f"inv_freq must be [rot_dim / 2] with rot_dim from 2 to {D}")
    if not rope_scale > 0:
        raise ValueError("rope_scale must be above 0")
    qw = kw = None
    if q_weight is not None:
        qw = _flat(q_weight, "q_weight", _BF16, dev)
        if q_weight.shape != (D,):
            raise ValueError(f"q_weight must be [{D}]")
    if k_weight is not None:
        kw = _flat(k_weight, "k_weight", _BF16, dev)
        if k_weight.shape != (D,):
            raise ValueError(f"k_weight must be [{D}]")
    return Rope(f, 2 * inv_freq.shape[0], 1 if interleaved else 0, rope_scale, qw, kw, eps)


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, rope_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Norm (where there are weights) and rotation of query and key heads.

    q [N][Hq][D] and k [N][Hkv][D] with positions int32 [N], or
    [B][Hq][T][D] and [B][Hkv][T][D] with positions [B][T]; bf16 views of any
    strides whose heads are contiguous, so slices of a projection's rows are
    taken as they are.  inv_freq fp32 [rot_dim/2]: the first rot_dim values of
    a head are turned, as pairs (i, i + rot_dim/2) or, interleaved,
    (2i, 2i + 1).  For contexts stretched beyond training pass the stretched
    frequencies and, as rope_scale, the factor on cos and sin that goes with
    them.  Returns (q_out, k_out), contiguous unless given; q_out=q, k_out=k
    works in place."""
    dev, shape, ks = q.get_device(), q.shape, k.shape
    if len(shape) == 3 and len(ks) == 3:
        (T, Hq, D), B, Hkv, b, n, h = shape, 1, ks[1], -1, 0, 1
        same, want = ks[0] == T, (T,)
    elif len(shape) == 4 and len(ks) == 4:
        (B, Hq, T, D), Hkv, b, n, h = shape, ks[1], 0, 2, 1
        same, want = ks[0] == B and ks[2] == T, (B, T)
    else:
        raise ValueError("q and k must be [N][H][D] or [B][H][T][D]")
    if not same or ks[-1] != D:
        raise ValueError(f"q {list(shape)} and k {list(ks)} do not belong together")
    pos = _flat(positions, "positions", _I32, dev)
    if positions.shape != want:
        raise ValueError(f"positions must be {list(want)}, got {list(positions.shape)}")
    rope = _rope(inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, D, dev)
    st = _stream_on(dev, stream)
    if q_out is None:
        q_out = _like(q, stream)
    elif q_out.shape != shape:
        raise ValueError(f"q_out must be {list(shape)}")
    if k_out is None:
        k_out = _like(k, stream)
    elif k_out.shape != ks:
        raise ValueError(f"k_out must be {list(ks)}")
    _check((_lib or load()).longspec_hta_qk_norm_rope(
        B, T, Hq, Hkv, D, _heads(q, "q", dev, b, n, h), _heads(k, "k", dev, b, n, h), pos, rope,
        _heads(q_out, "q_out", dev, b, n, h), _heads(k_out, "k_out", dev, b, n, h), st))
    return q_out, k_out


def _ragged(prefix_len, q_start, block_table, dev: int):
    pre, start = _flat(prefix_len, "prefix_len", _I32, dev), _flat(q_start, "q_start", _I32, dev)
    B = prefix_len.shape[0] if prefix_len.dim() == 1 else 0
    if B < 1 or q_start.shape != (B + 1,) or block_table.shape[0] != B:
        raise ValueError("prefix_len must be [B], q_start [B + 1], block_table [B][max_blocks]")
    return B, pre, start


def _append(q, k, v, rope, k_cache, v_cache, block_table, prefix_len, q_start, L_cap, k_scale, v_scale, q_out,
            workspace, stream):
    dev = k.get_device()
    N, Hkv, D = k.shape
    if v.shape != k.shape or (q is not None and (q.dim() != 3 or q.shape[0] != N or q.shape[2] != D)):
        raise ValueError("k and v must be [N][Hkv][D], q [N][Hq][D]")
    if k_cache.dim() != 4 or k_cache.shape[1] != Hkv or k_cache.shape[3] != D:
        raise ValueError(f"the cache must be [num_blocks][{Hkv}][block_size][{D}]")
    cache = _cache(k_cache, v_cache, block_table, k_scale, v_scale, dev)
    B, pre, start = _ragged(prefix_len, q_start, block_table, dev)
    st = _stream_on(dev, stream)
    Hq, qh, oh = Hkv, None, None
    if q is not None:
        Hq = q.shape[1]
        if q_out is None:
            q_out = _like(q, stream)
        elif q_out.shape != q.shape:
            raise ValueError(f"q_out must be {list(q.shape)}")
        qh, oh = _heads(q, "q", dev, -1, 0, 1), _heads(q_out, "q_out", dev, -1, 0, 1)
    if workspace is None:
        workspace = _new(stream, torch.zeros, 256, dtype=torch.uint8, device=k.device)
    _check((_lib or load()).longspec_hta_append_paged(
        Dims(B, Hq, Hkv, D, N, L_cap, 0.0), qh, _heads(k, "k", dev, -1, 0, 1), _heads(v, "v", dev, -1, 0, 1), rope,
        cache, pre, start, oh, _flat(workspace, "workspace", torch.uint8, dev), workspace.nbytes, st))
    return q_out


def append_paged(k, v, k_cache, v_cache, block_table, prefix_len, q_start, *, L_cap, k_scale=None, v_scale=None,
                 workspace=None, stream=None):
    """Append new tokens' K/V rows [N][Hkv][D] (views of any strides whose
    heads are contiguous) to a paged cache: rows q_start[b] .. q_start[b+1]-1
    go to positions prefix_len[b] .. of sequence b (q_start int32 [B+1],
    ascending; rows from q_start[B] on are padding).  prefix_len is not
    advanced.

    The cache is bf16, or e4m3 with a scale byte e per row in k_scale and
    v_scale (uint8 [num_blocks][Hkv][block_size]): a row is kept as codes
    times 2^(e - 127), the smallest power of two under which the row's
    largest value stays within 448 (e clamped to [16, 134]; a row with an
    infinity or a NaN reads back as NaN).  Problems on the device
    (lengths past L_cap, bad blocks, ranges out of order) leave those rows
    unwritten and show in get_status(workspace); workspace: at least 256
    bytes, zeroed."""
    _append(None, k, v, None, k_cache, v_cache, block_table, prefix_len, q_start, L_cap, k_scale, v_scale, None,
            workspace, stream)


def rope_append_paged(q, k, v, inv_freq, k_cache, v_cache, block_table, prefix_len, q_start, *, L_cap,
                      q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                      rope_scale: float = 1.0, k_scale=None, v_scale=None, q_out=None, workspace=None,
                      stream=None):
    """append_paged() with the norm and rotation of qk_norm_rope() in the same
    pass: q and k are normed and rotated at their positions
    prefix_len[b] + place in the chunk, k and v go to the cache.  Returns
    q_out [N][Hq][D]; padding rows of it are left as they were."""
    rope = _rope(inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, k.shape[-1], k.get_device())
    return _append(q, k, v, rope, k_cache, v_cache, block_table, prefix_len, q_start, L_cap, k_scale, v_scale, q_out,
                   workspace, stream)


def new_chunk_workspace(q, k_cache, B: int, *, L_cap: int) -> torch.Tensor:
    """A zeroed workspace for chunk_attention_paged calls of q's shape."""
    N, Hq, D = q.shape
    n = load().longspec_hta_chunk_workspace_bytes(Dims(B, Hq, k_cache.shape[1], D, N, L_cap, 0.0))
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def chunk_attention_paged(q, k_cache, v_cache, block_table, prefix_len, q_start, *, L_cap, window: int = 0,
                          k_scale=None, v_scale=None, scale: float = 0.0, out=None, lse=None, workspace=None,
                          stream=None):
    """Causal attention of chunks of new tokens over the paged cache that
    holds them (append_paged / rope_append_paged before this call).

    q [N][Hq][D] bf16 (tokens at any stride): rows q_start[b] ..
    q_start[b+1]-1 are at positions prefix_len[b] .. of sequence b and attend
    to its keys up to their own position, to the last `window` of them when
    window > 0.  Single tokens (a decode step), whole prompts and ragged
    mixtures are all such chunks.  The cache is bf16, or e4m3 with scales.
    Returns (out bf16 [N][Hq][D], lse fp32 [N][Hq]); padding rows (from
    q_start[B] on) are left as they were."""
    dev = q.get_device()
    N, Hq, D = shape = q.shape
    if k_cache.dim() != 4 or k_cache.shape[3] != D or Hq % k_cache.shape[1]:
        raise ValueError(f"the cache must be [num_blocks][Hkv][block_size][{D}] with Hkv dividing {Hq}")
    cache = _cache(k_cache, v_cache, block_table, k_scale, v_scale, dev)
    B, pre, start = _ragged(prefix_len, q_start, block_table, dev)
    st = _stream_on(dev, stream)
    if Hq > 1 and q.stride(1) != D:
        raise ValueError("q: the heads of a token must be contiguous")
    out = _like(q, stream) if out is None else _result(out, "out", shape, _BF16, dev)
    lse = (_new(stream, q.new_empty, (N, Hq), dtype=torch.float32) if lse is None
           else _result(lse, "lse", (N, Hq), torch.float32, dev))
    if workspace is None:
        workspace = _new(stream, new_chunk_workspace, q, k_cache, B, L_cap=L_cap)
    _check((_lib or load()).longspec_hta_chunk_attention_paged(
        Dims(B, Hq, k_cache.shape[1], D, N, L_cap, scale), _heads(q, "q", dev, -1, 0, 1), cache, pre, start, window,
        out.data_ptr(), lse.data_ptr(), _flat(workspace, "workspace", torch.uint8, dev), workspace.nbytes, st))
    return out, lse


def _attention_q8(q, k_cache, v_cache, block_table, prefix_len, tree, L_cap, out, lse, workspace, scale, num_splits,
                  prefix_events, stream, k_scale, v_scale):
    """verify_paged (tree: k_tree, v_tree, parent) or prefix_attention_paged
    over an e4m3 cache."""
    if num_splits or prefix_events:
        raise ValueError("num_splits and prefix_events do not apply to an e4m3 cache")
    dev, shape = q.get_device(), q.shape
    qp, pre = _flat(q, "q", _BF16, dev), _flat(prefix_len, "prefix_len", _I32, dev)
    cache = _cache(k_cache, v_cache, block_table, k_scale, v_scale, dev)
    dims = _paged_dims(q, k_cache, L_cap, scale)
    kt, vt, parent = tree or (None, None, None)
    _tree_shapes(dims, k_cache, prefix_len, block_table, kt, vt, parent)
    st = _stream_on(dev, stream)
    out = _like(q, stream) if out is None else _result(out, "out", shape, _BF16, dev)
    lse = (_new(stream, q.new_empty, shape[:3], dtype=torch.float32) if lse is None
           else _result(lse, "lse", shape[:3], torch.float32, dev))
    workspace = _new(stream, new_q8_workspace, dims, q.device) if workspace is None else workspace
    end = (out.data_ptr(), lse.data_ptr(), _flat(workspace, "workspace", torch.uint8, dev), workspace.nbytes, st)
    lib = _lib or load()
    if tree is None:
        _check(lib.longspec_hta_prefix_attention_paged_q8(dims, qp, cache, pre, *end))
    else:
        _check(lib.longspec_hta_verify_paged_q8(dims, qp, cache, pre, _flat(kt, "k_tree", _BF16, dev),
                                                _flat(vt, "v_tree", _BF16, dev), _flat(parent, "parent", _I32, dev),
                                                *end))
    return out, lse


def new_q8_workspace(dims: Dims, device=None) -> torch.Tensor:
    """A zeroed workspace for verify_paged / prefix_attention_paged over an
    e4m3 cache."""
    n = load().longspec_hta_q8_workspace_bytes(dims)
    if n == 0:
        raise HtaError(ERR_INVALID_DIMS)
    return torch.zeros(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def selftest_wait_timeout(workspace: torch.Tensor, stream=None) -> int:
    """Launch the failure-detection self-test on `workspace`'s status word:
    one bounded in-kernel wait that nothing completes (about 2 s); a later
    get_status() returns ERR_PIPELINE_TIMEOUT."""
    return int(load().longspec_hta_selftest_wait_timeout(_ptr(workspace), _stream(stream)))


def build_info() -> dict:
    """The loaded library's build-time tuning knobs, e.g.
    {"kv_stages_d128": 3, "exp2_poly_every": 4}."""
    text = load().longspec_hta_build_info().decode()
    return {k: int(v) for k, v in (kv.split("=") for kv in text.split())}


def get_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise, read and clear the device status word; returns the code."""
    return int(load().longspec_hta_get_status(_ptr(workspace), _stream(stream)))
