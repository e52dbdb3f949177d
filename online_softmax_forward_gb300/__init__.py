"""Python binding of libattn.so -- exact attention forward with online softmax
for GB300 (sm_103a).

The functions named like the C ABI (``attn_fwd``, ``attn_validate``, ...)
take raw pointers and sizes and only marshal arguments; ``attention`` is the
convenience call on PyTorch CUDA tensors (it allocates the outputs with torch
and calls ``attn_fwd``).  Every step of the computation runs in the library's
CUDA kernels; if the library is missing this module raises instead of
computing anything another way.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

__all__ = [
    "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED_DEVICE", "ATTN_ERR_LAUNCH",
    "ATTN_ERR_TIMEOUT", "ATTN_ERR_CUDA", "ATTN_ERR_SCRATCH_LIMIT", "ATTN_ERR_BOUNDS",
    "ATTN_ERR_TABLE", "ATTN_CACHE_E4M3", "ATTN_CACHE_I8",
    "NOALLOC_SCRATCH_BYTES",
    "ATTN_F32", "ATTN_BF16", "ATTN_F16", "ATTN_BF16_OUT_F32", "ATTN_F16_OUT_F32",
    "AttnError", "library_path", "load_library", "exported_symbols",
    "test_library_path", "load_test_library", "test_exported_symbols",
    "checked_library_path", "load_checked_library",
    "attn_fwd", "attn_validate", "attn_fwd_f32_blocked", "attn_fwd_staged",
    "attn_check_status", "attn_strerror", "attn_abi_version", "attn_test_set_hook",
    "attn_splitkv_workspace_size", "attn_splitkv_plan", "attn_fwd_splitkv", "attn_merge",
    "attn_fwd_splitkv_noalloc", "attn_shutdown",
    "attn_cache_append", "attn_cache_read", "attn_cache_select_workspace_size",
    "attn_cache_select", "attn_fwd_cache_workspace_size", "attn_fwd_cache",
    "attention", "attention_f32_blocked", "attention_splitkv", "merge", "dtype_code",
    "KVCache", "cache_append", "cache_read", "cache_select", "attention_cache",
]

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED_DEVICE = 2
ATTN_ERR_LAUNCH = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_CUDA = 5
ATTN_ERR_SCRATCH_LIMIT = 6
ATTN_ERR_BOUNDS = 7  # the bounds-checking build (libattn_checked.so) only
ATTN_ERR_TABLE = 8
NOALLOC_SCRATCH_BYTES = 8 << 20  # the fixed scratch of attn_fwd_splitkv_noalloc

ATTN_F32 = 0
ATTN_BF16 = 1
ATTN_F16 = 2
ATTN_BF16_OUT_F32 = 3
ATTN_F16_OUT_F32 = 4

ATTN_CACHE_E4M3 = 0
ATTN_CACHE_I8 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None
_test_lib = None
_checked_lib = None

# (name, restype, argtypes) of every symbol declared in include/attn.h
# (libattn.so) and, in _TEST_SIGS, in include/attn_test.h (libattn_test.so only)
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t


class _Cache(ctypes.Structure):  # attn_cache of include/attn.h
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("k_bounds", _P),
                ("n_pages", _I), ("H_kv", _I), ("page", _I), ("d", _I), ("format", _I)]


_C = ctypes.POINTER(_Cache)
_SIGS = [
    ("attn_fwd", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    ("attn_validate", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I]),
    ("attn_fwd_staged", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                             _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    ("attn_check_status", _I, [_P]),
    ("attn_strerror", ctypes.c_char_p, [_I]),
    ("attn_abi_version", _I, []),
    ("attn_splitkv_workspace_size", _I, [_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    ("attn_splitkv_plan", _I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(_I),
                               ctypes.POINTER(ctypes.c_size_t)]),
    ("attn_fwd_splitkv", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P,
                              ctypes.c_size_t, _P]),
    ("attn_merge", _I, [_P, _P, _I, ctypes.c_int64, _I, _P, _P, _I, _P]),
    ("attn_fwd_splitkv_noalloc", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                                      _P]),
    ("attn_shutdown", _I, []),
    ("attn_cache_append", _I, [_C, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P]),
    ("attn_cache_read", _I, [_C, _P, _I, _P, _P, _P, _I, _I, _I, _P]),
    ("attn_cache_select_workspace_size", _I, [_I, _I, _I, _I, ctypes.POINTER(_Z)]),
    ("attn_cache_select", _I, [_C, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z, _P]),
    ("attn_fwd_cache_workspace_size", _I, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_Z)]),
    ("attn_fwd_cache", _I, [_C, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _Z,
                            _P]),
]
_TEST_SIGS = [
    ("attn_fwd_f32_blocked", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    ("attn_test_set_hook", _I, [_I, ctypes.c_uint64]),
]


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, _strerror_safe(status), status))


def library_path() -> str:
    return os.environ.get("ATTN_GB300_LIB", os.path.join(_HERE, "libattn.so"))


def test_library_path() -> str:
    return os.environ.get("ATTN_GB300_TEST_LIB", os.path.join(_HERE, "libattn_test.so"))


def _open(path, sigs, what):
    if not os.path.exists(path):
        raise ImportError("%s not found at %s: build it with "
                          "online_softmax_forward_gb300.build.build()" % (what, path))
    lib = ctypes.CDLL(path)
    for name, res, args in sigs:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load_library():
    """Load libattn.so (built by ``build.build()``); raises if it is absent."""
    global _lib
    if _lib is None:
        _lib = _open(library_path(), _SIGS, "libattn.so")
    return _lib


def load_test_library():
    """Load libattn_test.so: the product's functions plus the test-only entry
    points of include/attn_test.h.  It is a separate library with its own
    state (status word, hook): call the functions of a test on it alone."""
    global _test_lib
    if _test_lib is None:
        _test_lib = _open(test_library_path(), _SIGS + _TEST_SIGS, "libattn_test.so")
    return _test_lib


def checked_library_path() -> str:
    return os.path.join(_HERE, "libattn_checked.so")


def load_checked_library():
    """Load libattn_checked.so: the test library built with ATTN_BOUNDS_CHECK,
    whose kernels test every global index and TMA coordinate before using it
    (attn_check_status then reports ATTN_ERR_BOUNDS).  A separate library
    with its own state, like the test library."""
    global _checked_lib
    if _checked_lib is None:
        _checked_lib = _open(checked_library_path(), _SIGS + _TEST_SIGS, "libattn_checked.so")
    return _checked_lib


def exported_symbols():
    return [s[0] for s in _SIGS]


def test_exported_symbols():
    return [s[0] for s in _TEST_SIGS]


def _strerror_safe(status: int) -> str:
    try:
        return load_library().attn_strerror(int(status)).decode()
    except Exception:  # pragma: no cover
        return "status %d" % status


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)
    return status


# ------------------------------------------------------------------ raw ABI
def attn_fwd(q, k, v, o, lse, B, H, Sq, Skv, d, causal, scale, dtype, stream):
    return load_library().attn_fwd(q, k, v, o, lse, B, H, Sq, Skv, d, int(causal),
                                   float(scale), dtype, stream)


def attn_validate(q, k, v, o, lse, B, H, Sq, Skv, d, causal, scale, dtype):
    return load_library().attn_validate(q, k, v, o, lse, B, H, Sq, Skv, d, int(causal),
                                        float(scale), dtype)


def attn_fwd_f32_blocked(q, k, v, o, lse, B, H, Sq, Skv, d, causal, scale, block_q,
                         block_kv, stream):
    """Test library only (include/attn_test.h)."""
    return load_test_library().attn_fwd_f32_blocked(q, k, v, o, lse, B, H, Sq, Skv, d,
                                                    int(causal), float(scale), block_q,
                                                    block_kv, stream)


def attn_fwd_staged(q_host, k_host, v_host, o_host, lse_host, dq, dk, dv, do_, dlse,
                    B, H, Sq, Skv, d, causal, scale, dtype, stream):
    return load_library().attn_fwd_staged(q_host, k_host, v_host, o_host, lse_host, dq, dk,
                                           dv, do_, dlse, B, H, Sq, Skv, d, int(causal),
                                           float(scale), dtype, stream)


def attn_check_status(stream):
    return load_library().attn_check_status(stream)


def attn_strerror(status):
    return load_library().attn_strerror(int(status)).decode()


def attn_abi_version():
    return load_library().attn_abi_version()


def attn_shutdown():
    return load_library().attn_shutdown()


def attn_test_set_hook(hook, timeout_ns=0):
    """Test library only (include/attn_test.h): arms the hook of
    libattn_test.so, which affects that library's attn_fwd alone."""
    return load_test_library().attn_test_set_hook(int(hook), int(timeout_ns))


def attn_splitkv_workspace_size(B, H, Sq, d, n_splits):
    """Returns (status, bytes)."""
    n = ctypes.c_size_t(0)
    st = load_library().attn_splitkv_workspace_size(B, H, Sq, d, n_splits, ctypes.byref(n))
    return st, n.value


def attn_splitkv_plan(B, H, Sq, Skv, d, dtype):
    """Returns (status, n_splits, workspace_bytes)."""
    n = ctypes.c_int(0)
    b = ctypes.c_size_t(0)
    st = load_library().attn_splitkv_plan(B, H, Sq, Skv, d, dtype, ctypes.byref(n),
                                          ctypes.byref(b))
    return st, n.value, b.value


def attn_fwd_splitkv(q, k, v, o, lse, B, H, Sq, Skv, d, causal, scale, dtype, n_splits,
                     workspace, workspace_bytes, stream):
    return load_library().attn_fwd_splitkv(q, k, v, o, lse, B, H, Sq, Skv, d, int(causal),
                                           float(scale), dtype, int(n_splits), workspace,
                                           int(workspace_bytes), stream)


def attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, H, Sq, Skv, d, causal, scale, dtype, n_splits,
                             stream):
    """attn_fwd_splitkv with the library's fixed device scratch instead of a
    workspace: for callers that cannot allocate (see include/attn.h)."""
    return load_library().attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, H, Sq, Skv, d,
                                                   int(causal), float(scale), dtype,
                                                   int(n_splits), stream)


def attn_merge(o_parts, lse_parts, n_parts, rows, d, o, lse, out_dtype, stream):
    return load_library().attn_merge(o_parts, lse_parts, int(n_parts), int(rows), int(d), o,
                                     lse, int(out_dtype), stream)


def attn_cache_append(cache, k, v, table, max_pages, pos, counts, B, S, dtype, stream):
    """``cache`` is a _Cache structure (KVCache.c)."""
    return load_library().attn_cache_append(cache, k, v, table, max_pages, pos, counts, B, S,
                                            dtype, stream)


def attn_cache_read(cache, table, max_pages, lens, k, v, B, S, dtype, stream):
    return load_library().attn_cache_read(cache, table, max_pages, lens, k, v, B, S, dtype, stream)


def attn_cache_select_workspace_size(B, H_kv, Sq, max_pages):
    """Returns (status, bytes)."""
    n = _Z(0)
    st = load_library().attn_cache_select_workspace_size(B, H_kv, Sq, max_pages, ctypes.byref(n))
    return st, n.value


def attn_cache_select(cache, q, table, max_pages, lens, counts, pages, n_select, B, H, Sq, causal,
                      dtype, workspace, workspace_bytes, stream):
    return load_library().attn_cache_select(cache, q, table, max_pages, lens, counts, pages,
                                            n_select, B, H, Sq, int(causal), dtype, workspace,
                                            int(workspace_bytes), stream)


def attn_fwd_cache_workspace_size(B, H, H_kv, Sq, d, dtype, n_select=0):
    """Returns (status, bytes)."""
    n = _Z(0)
    st = load_library().attn_fwd_cache_workspace_size(B, H, H_kv, Sq, d, dtype, n_select,
                                                      ctypes.byref(n))
    return st, n.value


def attn_fwd_cache(cache, q, o, lse, table, max_pages, lens, counts, pages, n_select, B, H, Sq,
                   causal, scale, dtype, workspace, workspace_bytes, stream):
    return load_library().attn_fwd_cache(cache, q, o, lse, table, max_pages, lens, counts, pages,
                                         n_select, B, H, Sq, int(causal), float(scale), dtype,
                                         workspace, int(workspace_bytes), stream)


# ------------------------------------------------------------------ torch helpers
def dtype_code(in_dtype, out_dtype=None) -> int:
    """attn_dtype for torch input/output dtypes."""
    import torch
    if in_dtype == torch.float32:
        if out_dtype not in (None, torch.float32):
            raise ValueError("fp32 inputs give fp32 output")
        return ATTN_F32
    if in_dtype == torch.bfloat16:
        if out_dtype in (None, torch.bfloat16):
            return ATTN_BF16
        if out_dtype == torch.float32:
            return ATTN_BF16_OUT_F32
    if in_dtype == torch.float16:
        if out_dtype in (None, torch.float16):
            return ATTN_F16
        if out_dtype == torch.float32:
            return ATTN_F16_OUT_F32
    raise ValueError("unsupported dtypes %s -> %s" % (in_dtype, out_dtype))


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, S, d]")
    B, H, Sq, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != H or k.shape[3] != d:
        raise ValueError("shape mismatch q %s k %s v %s" % (tuple(q.shape), tuple(k.shape),
                                                            tuple(v.shape)))
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    _device_of(q, k, v)
    return B, H, Sq, k.shape[2], d


def _device_of(*tensors):
    """The one CUDA device all tensors live on; raises otherwise (the kernels
    are handed raw device pointers)."""
    dev = None
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors (got %s)" % t.device)
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors on different devices: %s and %s" % (dev, t.device))
    return dev


def _check_out(t, shape, dtype, dev, name):
    """A caller-provided output must match exactly what the call writes."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
    if not t.is_cuda or t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))


def attention(q, k, v, causal: bool = False, scale: float | None = None, out_dtype=None,
              return_lse: bool = True, out=None, lse=None, stream=None):
    """O (and LSE) for contiguous CUDA tensors q [B,H,Sq,d], k/v [B,H,Skv,d].

    ``out_dtype`` = torch.float32 with bf16/fp16 inputs selects the fp32-output
    variant.  Outputs are allocated with torch unless ``out`` / ``lse`` are
    given."""
    import torch
    B, H, Sq, Skv, d = _shapes(q, k, v)
    code = dtype_code(q.dtype, out_dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share a dtype")
    odt = {ATTN_F32: torch.float32, ATTN_BF16: torch.bfloat16, ATTN_F16: torch.float16,
           ATTN_BF16_OUT_F32: torch.float32, ATTN_F16_OUT_F32: torch.float32}[code]
    if out is None:
        out = torch.empty((B, H, Sq, d), dtype=odt, device=q.device)
    _check_out(out, (B, H, Sq, d), odt, q.device, "out")
    if return_lse and lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_out(lse, (B, H, Sq), torch.float32, q.device, "lse")
    sc = 0.0 if scale is None else float(scale)
    with torch.cuda.device(q.device):
        st = attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                      lse.data_ptr() if lse is not None else None, B, H, Sq, Skv, d, causal,
                      sc, code, _stream_handle(stream))
    _check(st, "attn_fwd")
    return (out, lse) if return_lse else out


def attention_f32_blocked(q, k, v, block_q: int, block_kv: int, causal: bool = False,
                          scale: float | None = None, stream=None):
    """fp32 path with explicit tile sizes (block-size invariance tests;
    runs in the test library, include/attn_test.h)."""
    import torch
    B, H, Sq, Skv, d = _shapes(q, k, v)
    out = torch.empty((B, H, Sq, d), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    with torch.cuda.device(q.device):
        st = attn_fwd_f32_blocked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, H, Sq, Skv, d, causal, sc, block_q,
                                  block_kv, _stream_handle(stream))
    _check(st, "attn_fwd_f32_blocked")
    return out, lse


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def attention_splitkv(q, k, v, causal: bool = False, scale: float | None = None,
                      out_dtype=None, n_splits: int | None = None, workspace=None,
                      stream=None):
    """Split-KV forward (few query rows, long key sequences).  The workspace is
    a torch uint8 CUDA tensor, allocated here unless given; ``n_splits`` is
    the library's choice unless given.  Returns (o, lse)."""
    import torch
    B, H, Sq, Skv, d = _shapes(q, k, v)
    code = dtype_code(q.dtype, out_dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share a dtype")
    if n_splits is None:
        with torch.cuda.device(q.device):
            st, n_splits, _ = attn_splitkv_plan(B, H, Sq, Skv, d, code)
        _check(st, "attn_splitkv_plan")
    st, need = attn_splitkv_workspace_size(B, H, Sq, d, n_splits)
    _check(st, "attn_splitkv_workspace_size")
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if not workspace.is_contiguous() or _device_of(workspace) != q.device:
        raise ValueError("workspace must be a contiguous tensor on %s" % q.device)
    odt = {ATTN_F32: torch.float32, ATTN_BF16: torch.bfloat16, ATTN_F16: torch.float16,
           ATTN_BF16_OUT_F32: torch.float32, ATTN_F16_OUT_F32: torch.float32}[code]
    out = torch.empty((B, H, Sq, d), dtype=odt, device=q.device)
    lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    sc = 0.0 if scale is None else float(scale)
    with torch.cuda.device(q.device):
        st = attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr(), B, H, Sq, Skv, d, causal, sc, code, n_splits,
                              workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                              _stream_handle(stream))
    _check(st, "attn_fwd_splitkv")
    return out, lse


def merge(o_parts, lse_parts, out_dtype=None, stream=None):
    """attn_merge on torch tensors: o_parts [n, rows, d] fp32, lse_parts
    [n, rows] fp32 -> (o [rows, d], lse [rows])."""
    import torch
    if o_parts.dim() != 3 or lse_parts.shape != o_parts.shape[:2]:
        raise ValueError("o_parts [n, rows, d] and lse_parts [n, rows] expected")
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise ValueError("partial results are fp32")
    o_parts, lse_parts = o_parts.contiguous(), lse_parts.contiguous()
    _device_of(o_parts, lse_parts)
    n, rows, d = o_parts.shape
    odt = torch.float32 if out_dtype is None else out_dtype
    code = {torch.float32: ATTN_F32, torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}[odt]
    out = torch.empty((rows, d), dtype=odt, device=o_parts.device)
    lse = torch.empty((rows,), dtype=torch.float32, device=o_parts.device)
    with torch.cuda.device(o_parts.device):
        st = attn_merge(o_parts.data_ptr(), lse_parts.data_ptr(), n, rows, d, out.data_ptr(),
                        lse.data_ptr(), code, _stream_handle(stream))
    _check(st, "attn_merge")
    return out, lse


# ------------------------------------------------------------------ paged 8-bit cache
class _Scratch(threading.local):
    """A thread's workspaces of one cache, which end with the thread."""

    def __init__(self):
        self.kept = {}  # stream handle -> workspace of the calls on it


class KVCache:
    """The pool of a paged 8-bit key/value cache (include/attn.h): five
    contiguous CUDA tensors the caller owns,

    ``k``, ``v`` [n_pages, H_kv, page, d] of torch.float8_e4m3fn or torch.int8,
    ``k_scale``, ``v_scale`` [n_pages, H_kv] fp32 and, for ``cache_select``,
    ``k_bounds`` [n_pages, H_kv, 2, d] of the codes' type.  The tensors may be
    read at any time; nothing in them needs to be initialised."""

    def __init__(self, k, v, k_scale, v_scale, k_bounds=None):
        import torch
        _bind(torch)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [n_pages, H_kv, page, d] of one dtype")
        formats = {torch.float8_e4m3fn: ATTN_CACHE_E4M3, torch.int8: ATTN_CACHE_I8}
        if k.dtype not in formats:
            raise ValueError("codes must be float8_e4m3fn or int8, got %s" % k.dtype)
        n, h, page, d = k.shape
        if page not in (16, 32, 64, 128) or d not in (64, 128):
            raise ValueError("page must be 16, 32, 64 or 128 and d 64 or 128, got %d and %d" % (page, d))
        if n < 1 or h < 1:
            raise ValueError("a pool has at least one page and one kv head, got %d and %d" % (n, h))
        dev = _device_of(k, v)
        for t, name in ((k, "k"), (v, "v")):
            _check_out(t, (n, h, page, d), k.dtype, dev, name)
        _check_out(k_scale, (n, h), torch.float32, dev, "k_scale")
        _check_out(v_scale, (n, h), torch.float32, dev, "v_scale")
        if k_bounds is not None:
            _check_out(k_bounds, (n, h, 2, d), k.dtype, dev, "k_bounds")
        self.k, self.v, self.k_scale, self.v_scale, self.k_bounds = k, v, k_scale, v_scale, k_bounds
        self.n_pages, self.H_kv, self.page, self.d = n, h, page, d
        self.device = k.device
        self._scratch = _Scratch()
        self.c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        k_bounds.data_ptr() if k_bounds is not None else None, n, h, page, d,
                        formats[k.dtype])

    @classmethod
    def empty(cls, n_pages, H_kv, page, d, dtype=None, device="cuda", bounds=True):
        """A pool allocated with torch; ``dtype`` float8_e4m3fn (default) or int8."""
        import torch
        dtype = torch.float8_e4m3fn if dtype is None else dtype
        new = lambda *s, t=dtype: torch.empty(s, dtype=t, device=device)  # noqa: E731
        return cls(new(n_pages, H_kv, page, d), new(n_pages, H_kv, page, d),
                   new(n_pages, H_kv, t=torch.float32), new(n_pages, H_kv, t=torch.float32),
                   new(n_pages, H_kv, 2, d) if bounds else None)


def _int32_on(t, shape, device, name):
    """Pointer of an int32 array of the call."""
    if t.dtype is not _int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s on %s"
                         % (name, tuple(shape), device))
    return t.data_ptr()


def _sequence_args(cache, table, lens, counts, B):
    """Checks the arrays of the call's sequences; returns the table's pointer and width, and the
    pointers of lens and counts."""
    shape = table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("table must be [B, max_pages] with B = %d" % B)
    dev = cache.device
    one = (B,)
    return (_int32_on(table, shape, dev, "table"), shape[1], _int32_on(lens, one, dev, "lens"),
            None if counts is None else _int32_on(counts, one, dev, "counts"))


# What every call on a cache needs of torch, bound once a KVCache exists: looking it up in each
# call takes as long as a small kernel.
_torch = _int32 = _raw_stream = _current_device = _capturing = None


def _bind(torch):
    global _torch, _int32, _raw_stream, _current_device, _capturing
    _torch, _int32 = torch, torch.int32
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    _capturing = torch._C._cuda_isCurrentStreamCapturing


def _call_on(device, fn, *args):
    """fn(*args) with ``device`` current; raises for a status other than ATTN_OK."""
    if _current_device() == device.index:
        st = fn(*args)
    else:
        with _torch.cuda.device(device):
            st = fn(*args)
    if st != ATTN_OK:
        raise AttnError(st, fn.__name__)


def _handle(device, stream):
    """The cudaStream_t of ``stream``, or of the device's current stream: asked for without
    making a Stream object, which takes longer than a launch."""
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        raise ValueError("the cache is on %s, the stream on %s" % (device, stream.device))
    return stream.cuda_stream


def _new(stream, shape, dtype, device):
    """An uninitialised tensor that belongs to ``stream`` if one is given: memory that the
    current stream's work still uses is then not handed to another stream's."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


def _new_like(stream, t):
    """The same for a tensor of a contiguous one's shape, type and device, in less time."""
    if stream is None:
        return _torch.empty_like(t)
    return _new(stream, t.shape, t.dtype, t.device)


def _cache_rows(cache, k, v):
    """(B, S, attn_dtype) of new rows."""
    shape = k.shape
    if len(shape) != 4 or shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, H_kv, S, d] of one dtype")
    B, H, S, d = shape
    if H != cache.H_kv or d != cache.d:
        raise ValueError("k has %d heads of width %d, the cache %d of %d" % (H, d, cache.H_kv, cache.d))
    for t in (k, v):
        if not t.is_contiguous() or t.device != cache.device:
            raise ValueError("k and v must be contiguous tensors on %s" % cache.device)
    return B, S, dtype_code(k.dtype)


def cache_append(cache, k, v, table, pos, counts=None, stream=None):
    """Quantises the first ``counts[b]`` (default: all S) rows of k, v
    [B, H_kv, S, d] into the cache behind the ``pos[b]`` tokens sequence b
    holds.  ``table`` [B, max_pages], ``pos`` and ``counts`` [B] are int32 CUDA
    tensors, read on the device."""
    B, S, code = _cache_rows(cache, k, v)
    t, width, p, n = _sequence_args(cache, table, pos, counts, B)
    _call_on(cache.device, load_library().attn_cache_append, cache.c, k.data_ptr(), v.data_ptr(), t,
             width, p, n, B, S, code, _handle(cache.device, stream))


def cache_read(cache, table, lens, S, dtype=None, out=None, stream=None):
    """The first S tokens of each sequence as (k, v) [B, H_kv, S, d] of
    ``dtype`` (fp32, bf16 or fp16; default bf16); rows from lens[b] on are
    zero.  ``out`` is a pair of tensors to write instead of new ones."""
    B = table.shape[0] if table.dim() == 2 else -1
    if S < 0:
        raise ValueError("S must not be negative, got %d" % S)
    t, width, n, _ = _sequence_args(cache, table, lens, None, B)
    dtype = _torch.bfloat16 if dtype is None else dtype
    code = dtype_code(dtype)
    shape = (B, cache.H_kv, S, cache.d)
    handle = _handle(cache.device, stream)
    if out is None:
        k = _new(stream, shape, dtype, cache.device)
        v = _new_like(stream, k)
    else:
        k, v = out
        _check_out(k, shape, dtype, cache.device, "out[0]")
        _check_out(v, shape, dtype, cache.device, "out[1]")
    _call_on(cache.device, load_library().attn_cache_read, cache.c, t, width, n, k.data_ptr(),
             v.data_ptr(), B, S, code, handle)
    return k, v


def _cache_q(cache, q):
    """(B, H, Sq) of queries."""
    shape = q.shape
    if len(shape) != 4 or shape[3] != cache.d or shape[1] % cache.H_kv != 0 or shape[1] == 0:
        raise ValueError("q must be [B, H, Sq, %d] with H a multiple of %d, got %s"
                         % (cache.d, cache.H_kv, tuple(shape)))
    if not q.is_contiguous() or q.device != cache.device:
        raise ValueError("q must be a contiguous tensor on %s" % cache.device)
    return shape[0], shape[1], shape[2]


_KEPT_BYTES = 32 << 20  # of one kept workspace; attention needs 21 MB at most


@functools.lru_cache(maxsize=4096)
def _need(size, *args):
    """Bytes of a workspace: ``size`` depends on its arguments alone."""
    st, need = size(*args)
    _check(st, size.__name__)
    return need


def _workspace(workspace, need, cache, stream, handle):
    """(pointer, bytes, tensor) of the scratch of one call; the tensor has to outlive the launch.
    A thread's calls on one stream follow one another, so the cache keeps a workspace for each
    thread and stream (a call's two kernels need not be adjacent when two threads share a
    stream), up to a size that every attention call fits; a call that is being captured, or on a
    stream that it names, gets one of its own, which belongs to the graph or to that stream."""
    if workspace is not None:
        if not workspace.is_contiguous() or _device_of(workspace) != cache.device:
            raise ValueError("workspace must be a contiguous tensor on %s" % cache.device)
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    keep = stream is None and need <= _KEPT_BYTES and not _capturing()
    if keep:
        scratch = cache._scratch.kept
        kept = scratch.get(handle)
        if kept is not None and kept[1] >= need:
            return kept
    workspace = _new(stream, max(need, 16), _torch.uint8, cache.device)
    new = (workspace.data_ptr(), max(need, 16), workspace)
    if keep:
        scratch[handle] = new
    return new


def cache_select(q, cache, table, lens, n_select, counts=None, causal: bool = True, workspace=None,
                 stream=None):
    """The ``n_select`` pages each query attends to (attn_cache_select): int32
    [B, H_kv, Sq, n_select], ascending, -1 where fewer are visible."""
    B, H, Sq = _cache_q(cache, q)
    if cache.k_bounds is None:
        raise ValueError("the cache keeps no k_bounds")
    if n_select < 1:
        raise ValueError("n_select must be at least 1, got %d" % n_select)
    t, width, p, n = _sequence_args(cache, table, lens, counts, B)
    code = dtype_code(q.dtype)
    handle = _handle(cache.device, stream)
    need = _need(attn_cache_select_workspace_size, B, cache.H_kv, Sq, width)
    wp, wn, held = _workspace(workspace, need, cache, stream, handle)
    pages = _new(stream, (B, cache.H_kv, Sq, n_select), _int32, cache.device)
    _call_on(cache.device, load_library().attn_cache_select, cache.c, q.data_ptr(), t, width, p, n,
             pages.data_ptr(), n_select, B, H, Sq, 1 if causal else 0, code, wp, wn, handle)
    return pages


def attention_cache(q, cache, table, lens, counts=None, causal: bool = True,
                    scale: float | None = None, out_dtype=None, pages=None, workspace=None,
                    stream=None):
    """Attention of q [B, H, Sq, d] over the cached tokens of each sequence, or
    over the pages of ``pages`` [B, H_kv, Sq, n] (``cache_select``).  The last
    ``counts[b]`` (default Sq) of the ``lens[b]`` tokens are the queries' own.
    The workspace is allocated here unless given.  Returns (o, lse)."""
    B, H, Sq = _cache_q(cache, q)
    t, width, p, n = _sequence_args(cache, table, lens, counts, B)
    code = dtype_code(q.dtype, out_dtype)
    listed, n_select = None, 0
    if pages is not None:
        n_select = pages.shape[-1] if pages.dim() == 4 else 0
        if n_select < 1:
            raise ValueError("pages must be [B, H_kv, Sq, n] and list at least one page")
        listed = _int32_on(pages, (B, cache.H_kv, Sq, n_select), cache.device, "pages")
    handle = _handle(cache.device, stream)
    need = _need(attn_fwd_cache_workspace_size, B, H, cache.H_kv, Sq, cache.d, code, n_select)
    wp, wn, held = _workspace(workspace, need, cache, stream, handle)
    dev = cache.device
    out = _new_like(stream, q) if out_dtype is None else _new(stream, q.shape, out_dtype, dev)
    lse = _new(stream, (B, H, Sq), _torch.float32, dev)
    _call_on(cache.device, load_library().attn_fwd_cache, cache.c, q.data_ptr(), out.data_ptr(),
             lse.data_ptr(), t, width, p, n, listed, n_select, B, H, Sq, 1 if causal else 0,
             0.0 if scale is None else float(scale), code, wp, wn, handle)
    return out, lse
