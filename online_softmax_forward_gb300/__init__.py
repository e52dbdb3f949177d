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
import fractions
import functools
import math
import os
import struct
import threading
import warnings

__all__ = [
    "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED_DEVICE", "ATTN_ERR_LAUNCH",
    "ATTN_ERR_TIMEOUT", "ATTN_ERR_CUDA", "ATTN_ERR_SCRATCH_LIMIT", "ATTN_ERR_BOUNDS",
    "ATTN_ERR_TABLE", "ATTN_CACHE_E4M3", "ATTN_CACHE_I8",
    "NOALLOC_SCRATCH_BYTES",
    "ATTN_F32", "ATTN_BF16", "ATTN_F16", "ATTN_BF16_OUT_F32", "ATTN_F16_OUT_F32",
    "AttnError", "library_path", "load_library", "exported_symbols",
    "test_library_path", "load_test_library", "test_exported_symbols",
    "checked_library_path", "load_checked_library",
    "attn_fwd", "attn_fwd_gqa", "attn_validate", "attn_fwd_f32_blocked", "attn_fwd_staged",
    "attn_check_status", "attn_strerror", "attn_abi_version", "attn_test_set_hook",
    "attn_splitkv_workspace_size", "attn_splitkv_plan", "attn_fwd_splitkv", "attn_merge",
    "attn_fwd_splitkv_noalloc", "attn_shutdown",
    "attn_cache_append", "attn_cache_read", "attn_cache_select_workspace_size",
    "attn_cache_select", "attn_fwd_cache_workspace_size", "attn_fwd_cache",
    "attn_bwd_workspace_size", "attn_bwd", "attn_rotary",
    "attention", "attention_bwd", "attention_f32_blocked", "attention_splitkv", "merge", "dtype_code",
    "Rotary", "rotary", "KVCache", "cache_append", "cache_read", "cache_select", "attention_cache",
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


class _Heads(ctypes.Structure):  # attn_heads of include/attn.h
    _fields_ = [("in_", _P), ("out", _P), ("H", _I), ("in_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3)]


_HEADS = struct.Struct("PPi4x6q").pack  # the same as bytes, in a fifth of the time
_C = ctypes.POINTER(_Cache)
_R = ctypes.POINTER(_Heads)
_SIGS = [
    ("attn_fwd", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    ("attn_fwd_gqa", _I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    ("attn_bwd_workspace_size", _I, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_Z)]),
    ("attn_bwd", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I,
                      _P, _Z, _P]),
    ("attn_rotary", _I, [_R, _R, _P, _I, _I, _F, _I, _P, _I, _I, _I, _I, _I, _P]),
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
    lib.rotary_packed = lib["attn_rotary"]  # takes its structures as bytes
    lib.rotary_packed.restype = _I
    lib.rotary_packed.argtypes = [ctypes.c_char_p, ctypes.c_char_p] + lib.attn_rotary.argtypes[2:]
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


def attn_fwd_gqa(q, k, v, o, lse, B, H, H_kv, Sq, Skv, d, causal, scale, dtype, stream):
    return load_library().attn_fwd_gqa(q, k, v, o, lse, B, H, H_kv, Sq, Skv, d, int(causal),
                                       float(scale), dtype, stream)


def attn_bwd_workspace_size(B, H, H_kv, Sq, Skv, d, causal, dtype):
    """Returns (status, bytes)."""
    n = _Z(0)
    st = load_library().attn_bwd_workspace_size(B, H, H_kv, Sq, Skv, d, int(causal), dtype,
                                                ctypes.byref(n))
    return st, n.value


def attn_bwd(q, k, v, o, lse, do, dlse, dq, dk, dv, B, H, H_kv, Sq, Skv, d, causal, scale, dtype,
             workspace, workspace_bytes, stream):
    return load_library().attn_bwd(q, k, v, o, lse, do, dlse, dq, dk, dv, B, H, H_kv, Sq, Skv, d,
                                   int(causal), float(scale), dtype, workspace,
                                   int(workspace_bytes), stream)


def attn_rotary(q, k, turns, width, interleaved, amplitude, transpose, pos, pos_per_token, B, S, d,
                dtype, stream):
    """``q`` and ``k`` are _Heads structures; ``k`` may be None."""
    return load_library().attn_rotary(q, k, turns, width, int(interleaved), float(amplitude),
                                      int(transpose), pos, int(pos_per_token), B, S, d, dtype,
                                      stream)


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


def _shapes(q, k, v, shared=False):
    """(B, H, Sq, Skv, d); ``shared`` allows fewer kv heads, a divisor of H."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, S, d]")
    B, H, Sq, d = q.shape
    H_kv = k.shape[1]
    fits = H_kv == H or (shared and 0 < H_kv < H and H % H_kv == 0)
    if k.shape != v.shape or k.shape[0] != B or not fits or k.shape[3] != d:
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
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
    if not t.is_cuda or t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))


def _no_graph(name, *tensors):
    """Says that autograd will not see what it would be expected to; ``name`` is the caller's."""
    for t in tensors:
        if t is not None and t.requires_grad:
            if _torch.is_grad_enabled():
                warnings.warn("%s records no gradient for tensors that require one: attention_bwd and rotary(..., "
                              "transpose=True) compute them; call it under torch.no_grad()" % name, stacklevel=3)
            return


def attention(q, k, v, causal: bool = False, scale: float | None = None, out_dtype=None,
              return_lse: bool = True, out=None, lse=None, stream=None):
    """O (and LSE) for contiguous CUDA tensors q [B,H,Sq,d], k/v [B,H,Skv,d]
    (or [B,H_kv,Skv,d], H a multiple of H_kv: H / H_kv consecutive query heads
    share a kv head).

    ``out_dtype`` = torch.float32 with bf16/fp16 inputs selects the fp32-output
    variant.  Outputs are allocated with torch unless ``out`` / ``lse`` are
    given; those of a call that names a ``stream`` belong to that stream.
    Nothing is recorded for autograd (``attention_bwd`` has the gradients)."""
    if _torch is None:
        import torch
        _bind(torch)
    B, H, Sq, Skv, d = _shapes(q, k, v, shared=True)
    H_kv = k.shape[1]
    dtype, dev = q.dtype, q.device
    code = dtype_code(dtype, out_dtype)
    if k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k, v must share a dtype")
    _no_graph("attention", q, k, v)
    odt = dtype if out_dtype is None else out_dtype
    handle = _handle(dev, stream)
    if out is not None:
        _check_out(out, (B, H, Sq, d), odt, dev, "out")
    elif odt is dtype:
        out = _new_like(stream, q)
    else:
        out = _new(stream, (B, H, Sq, d), odt, dev)
    if lse is not None:
        _check_out(lse, (B, H, Sq), _torch.float32, dev, "lse")
    elif return_lse:
        lse = _new(stream, (B, H, Sq), _torch.float32, dev)
    sc = 0.0 if scale is None else float(scale)
    lp = None if lse is None else lse.data_ptr()
    if H_kv == H:
        _call_on(dev, load_library().attn_fwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                 lp, B, H, Sq, Skv, d, 1 if causal else 0, sc, code, handle)
    else:
        _call_on(dev, load_library().attn_fwd_gqa, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                 lp, B, H, H_kv, Sq, Skv, d, 1 if causal else 0, sc, code, handle)
    return (out, lse) if return_lse else out


def attention_bwd(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None,
                  dlse=None, out=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of a loss, from its gradients ``do`` in o and ``dlse`` (default: zero)
    in lse; q, k, v, causal and scale as given to ``attention``, o and lse as it returned them.

    q, do [B,H,Sq,d] and k, v [B,H_kv,Skv,d] share a dtype; the gradients have o's dtype (fp32 if
    the forward pass ran with ``out_dtype`` = torch.float32).  They are allocated with torch unless
    ``out`` = (dq, dk, dv) is given; the workspace (attn_bwd_workspace_size) belongs to the call, or is
    one that this thread keeps for the stream where ``out`` is given and the call is not captured.
    Nothing is recorded for autograd."""
    if _torch is None:
        import torch
        _bind(torch)
    if out is None and workspace is None and stream is None:
        r = _fast().attention_bwd(q, k, v, o, lse, do, dlse, causal, 0.0 if scale is None else scale)
        if type(r) is tuple:
            return r
        if r is not None:
            raise AttnError(r, "attn_bwd")
    shape, kshape, dtype, odt, dev = q.shape, k.shape, q.dtype, o.dtype, q.device
    if len(shape) != 4 or len(kshape) != 4 or v.shape != kshape or o.shape != shape or do.shape != shape:
        raise ValueError("q, o, do must be [B, H, Sq, d] of one shape and k, v [B, H_kv, Skv, d] of one")
    B, H, Sq, d = shape
    H_kv, Skv = kshape[1], kshape[2]
    if kshape[0] != B or kshape[3] != d or H < 1 or H_kv < 1 or H % H_kv != 0:
        raise ValueError("shape mismatch q %s k %s" % (tuple(shape), tuple(kshape)))
    if k.dtype is not dtype or v.dtype is not dtype or do.dtype is not dtype:
        raise ValueError("q, k, v and do must share a dtype")
    if not q.is_cuda or k.device != dev or v.device != dev or o.device != dev or do.device != dev:
        raise ValueError("q, k, v, o and do must be CUDA tensors on one device")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and o.is_contiguous()
            and do.is_contiguous()):
        raise ValueError("q, k, v, o and do must be contiguous")
    code = _codes.get((dtype, odt))
    if code is None:
        code = dtype_code(dtype, odt)  # raises
    rows = (B, H, Sq)
    _check_out(lse, rows, _float32, dev, "lse")
    if dlse is not None:
        _check_out(dlse, rows, _float32, dev, "dlse")
    _no_graph("attention_bwd", q, k, v, o, lse, do, dlse)
    handle = _handle(dev, stream)
    if out is not None:
        dq, dk, dv = out
        for t, like, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, k, "dv")):
            _check_out(t, like.shape, odt, dev, name)
    elif odt is dtype:
        dq, dk, dv = _new_like(stream, q), _new_like(stream, k), _new_like(stream, k)
    else:
        dq, dk, dv = (_new(stream, s, odt, dev) for s in (shape, kshape, kshape))
    need = _need(attn_bwd_workspace_size, B, H, H_kv, Sq, Skv, d, bool(causal), code)
    wp, wn, held = None, 0, None
    if need or workspace is not None:
        wp, wn, held = _workspace(workspace, need, _keeper(dev), stream, handle)
    _call_on(dev, load_library().attn_bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
             lse.data_ptr(), do.data_ptr(), None if dlse is None else dlse.data_ptr(),
             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, H_kv, Sq, Skv, d, 1 if causal else 0,
             0.0 if scale is None else float(scale), code, wp, wn, handle)
    return dq, dk, dv


def attention_f32_blocked(q, k, v, block_q: int, block_kv: int, causal: bool = False,
                          scale: float | None = None, stream=None):
    """fp32 path with explicit tile sizes (block-size invariance tests;
    runs in the test library, include/attn_test.h)."""
    import torch
    if _torch is None:
        _bind(torch)
    B, H, Sq, Skv, d = _shapes(q, k, v)
    out = _new(stream, (B, H, Sq, d), torch.float32, q.device)
    lse = _new(stream, (B, H, Sq), torch.float32, q.device)
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
    if _torch is None:
        _bind(torch)
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
        workspace = _new(stream, max(need, 16), torch.uint8, q.device)
    if not workspace.is_contiguous() or _device_of(workspace) != q.device:
        raise ValueError("workspace must be a contiguous tensor on %s" % q.device)
    odt = {ATTN_F32: torch.float32, ATTN_BF16: torch.bfloat16, ATTN_F16: torch.float16,
           ATTN_BF16_OUT_F32: torch.float32, ATTN_F16_OUT_F32: torch.float32}[code]
    out = _new(stream, (B, H, Sq, d), odt, q.device)
    lse = _new(stream, (B, H, Sq), torch.float32, q.device)
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
    if _torch is None:
        _bind(torch)
    if o_parts.dim() != 3 or lse_parts.shape != o_parts.shape[:2]:
        raise ValueError("o_parts [n, rows, d] and lse_parts [n, rows] expected")
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise ValueError("partial results are fp32")
    dev = _device_of(o_parts, lse_parts)
    with _on(stream, dev):
        o_parts, lse_parts = o_parts.contiguous(), lse_parts.contiguous()
    n, rows, d = o_parts.shape
    odt = torch.float32 if out_dtype is None else out_dtype
    code = {torch.float32: ATTN_F32, torch.bfloat16: ATTN_BF16, torch.float16: ATTN_F16}[odt]
    out = _new(stream, (rows, d), odt, dev)
    lse = _new(stream, (rows,), torch.float32, dev)
    with torch.cuda.device(dev):
        st = attn_merge(o_parts.data_ptr(), lse_parts.data_ptr(), n, rows, d, out.data_ptr(),
                        lse.data_ptr(), code, _stream_handle(stream))
    _check(st, "attn_merge")
    return out, lse


# ------------------------------------------------------------------ rotary positions
_PI = fractions.Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


class Rotary:
    """The angles of rotary positions: pair i of the first ``width`` channels turns by theta_i per
    position, theta_i = base ** (-2 i / width) unless ``frequencies`` gives them.

    ``layout``: "half" (pairs i, i + width / 2) or "interleaved" (2i, 2i + 1).
    ``scaling`` stretches positions for contexts ``factor`` times as long as trained:
      "linear"  theta_i / factor;
      "base"    a base of base * factor ** (width / (width - 2)): the fastest pair stays, the
                slowest is stretched by factor;
      "parts"   pairs that turn more than ``fast`` times within the trained ``context`` stay, those
                that turn less than ``slow`` times are divided by factor, between them both are
                blended linearly; the amplitude is then 1 + 0.1 ln(factor).
    ``amplitude`` overrides the factor on both results.  The table of width / 2 angles is held on
    ``device`` as 64-bit fractions of a turn (include/attn.h)."""

    def __init__(self, width, base=10000.0, layout="half", scaling=None, factor=1.0, context=None,
                 slow=1.0, fast=32.0, frequencies=None, amplitude=None, device="cuda"):
        import torch
        _bind(torch)
        if width < 2 or width % 2 != 0:
            raise ValueError("width must be even and at least 2, got %d" % width)
        if layout not in ("half", "interleaved"):
            raise ValueError("layout must be \"half\" or \"interleaved\", got %r" % (layout,))
        if scaling not in (None, "linear", "base", "parts"):
            raise ValueError("scaling must be None, \"linear\", \"base\" or \"parts\", got %r" % (scaling,))
        if not (factor > 0 and math.isfinite(factor)) or not (base > 0 and math.isfinite(base)):
            raise ValueError("base and factor must be positive and finite")
        if frequencies is not None:
            if scaling is not None:
                raise ValueError("frequencies are given as they are: scaling must be None")
            theta = [float(t) for t in frequencies]
            if len(theta) != width // 2:
                raise ValueError("width %d takes %d frequencies, got %d" % (width, width // 2, len(theta)))
        else:
            if scaling == "base":
                if width < 4:
                    raise ValueError("scaling \"base\" takes a width of at least 4")
                base = base * factor ** (width / (width - 2))
            theta = [base ** (-2.0 * i / width) for i in range(width // 2)]
            if scaling == "linear":
                theta = [t / factor for t in theta]
            elif scaling == "parts":
                if context is None or context < 1 or not fast > slow:
                    raise ValueError("scaling \"parts\" takes the trained context and slow < fast")
                for i, t in enumerate(theta):
                    keep = (context * t / (2.0 * math.pi) - slow) / (fast - slow)
                    keep = min(1.0, max(0.0, keep))
                    theta[i] = t * (keep + (1.0 - keep) / factor)
                if amplitude is None:
                    amplitude = 1.0 + 0.1 * math.log(factor) if factor > 1.0 else 1.0
        if not all(math.isfinite(t) for t in theta):
            raise ValueError("frequencies must be finite")
        self.width, self.layout, self.frequencies = width, layout, tuple(theta)
        self.amplitude = 1.0 if amplitude is None else float(amplitude)
        if not math.isfinite(self.amplitude):
            raise ValueError("amplitude must be finite")
        # theta / 2 pi of a turn, exactly, in units of 2^-64; as int64, which torch has everywhere
        turns = [round(fractions.Fraction(t) * 2 ** 63 / _PI) % 2 ** 64 for t in theta]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns],
                                  dtype=torch.int64, device=device)
        self.device = self.turns.device
        self._args = (self.turns.data_ptr(), width, 1 if layout == "interleaved" else 0, self.amplitude,
                      self.device.index if self.turns.is_cuda else -1)


def _heads(x, out, name):
    """attn_heads (packed) of rows x [B, H, S, d] written to ``out``."""
    xb, xh, xs, xc = x.stride()
    ob, oh, os_, oc = out.stride()
    if xc != 1 or oc != 1:
        raise ValueError("the channels of %s must be contiguous" % name)
    return _HEADS(x.data_ptr(), out.data_ptr(), x.shape[1], xb, xh, xs, ob, oh, os_)


def _contiguous_like(stream, t):
    """An uninitialised contiguous tensor of a strided one's shape, type and device."""
    if stream is None:
        return _torch.empty_like(t, memory_format=_contiguous)
    return _new(stream, t.shape, t.dtype, t.device)


def rotary(q, k, rot, pos, transpose: bool = False, out=None, stream=None):
    """Rows q [B,H,S,d] and k [B,H_kv,S,d] (or None) turned by the positions of their tokens.

    ``rot`` is a Rotary; ``pos`` an int32 CUDA tensor, [B,S], or [B] with the position of each
    sequence's first row.  q and k may be views of any strides with contiguous channels, for example
    of a projection's [B,S,H,d].  ``transpose`` gives the gradient in q and k from the one in the
    results.  New results are contiguous [B,H,S,d], as ``attention`` and ``cache_append`` take them;
    ``out`` = (q', k') writes to other places, which may be q and k themselves.  Returns (q', k').
    Nothing is recorded for autograd."""
    if out is None and stream is None:
        r = _fast().rotary(q, k, pos, transpose, *rot._args)
        if type(r) is tuple:
            return r
        if r is not None:
            raise AttnError(r, "attn_rotary")
    shape, dev, dtype = q.shape, q.device, q.dtype
    if len(shape) != 4:
        raise ValueError("q must be [B, H, S, d]")
    B, _, S, d = shape
    if dev != rot.device or not q.is_cuda:
        raise ValueError("q is on %s, the angles on %s" % (dev, rot.device))
    turns, width, interleaved, amplitude, _ = rot._args
    if width > d:
        raise ValueError("rows have %d channels, %d are turned" % (d, width))
    code = _codes.get((dtype, dtype))
    if code is None:
        code = dtype_code(dtype)  # raises
    if k is not None:
        kshape = k.shape
        if k.dtype is not dtype or k.device != dev or len(kshape) != 4 or kshape[0] != B or \
                kshape[2] != S or kshape[3] != d:
            raise ValueError("k must be [%d, H_kv, %d, %d] of q's dtype and device" % (B, S, d))
    _no_graph("rotary", q, k)
    per_token = pos.dim() == 2
    p = _int32_on(pos, (B, S) if per_token else (B,), dev, "pos")
    handle = _handle(dev, stream)
    if out is None:
        qo = _contiguous_like(stream, q)
        ko = None if k is None else _contiguous_like(stream, k)
    else:
        qo, ko = out
        for t, like, name in ((qo, q, "out[0]"), (ko, k, "out[1]")):
            if (t is None) != (like is None) or \
                    (t is not None and (t.shape != like.shape or t.dtype is not dtype or t.device != dev)):
                raise ValueError("%s must be of the shape, dtype and device of its input" % name)
    _call_on(dev, load_library().rotary_packed, _heads(q, qo, "q"),
             None if k is None else _heads(k, ko, "k"), turns, width, interleaved, amplitude,
             1 if transpose else 0, p, 1 if per_token else 0, B, S, d, code, handle)
    return qo, ko


# ------------------------------------------------------------------ paged 8-bit cache
class _Scratch(threading.local):
    """A thread's workspaces of one cache or device, which end with the thread."""

    def __init__(self):
        self.kept = {}  # stream handle -> workspace of the calls on it


class _Keeper:
    """What calls without an object of their own keep on a device."""

    def __init__(self, device):
        self.device, self._scratch = device, _Scratch()


_keepers = {}  # torch.device -> _Keeper


def _keeper(device):
    return _keepers.get(device) or _keepers.setdefault(device, _Keeper(device))


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
_calls = None  # module of csrc/torch_calls.cpp
_torch = _int32 = _float32 = _contiguous = _raw_stream = _current_device = _capturing = None
_codes = {}  # (input dtype, output dtype) -> attn_dtype


class _NoCalls:
    """In place of _torch_calls where it was not built (build.py): the wrappers' Python code does it all."""

    @staticmethod
    def rotary(*args):
        return None

    attention_bwd = rotary


def _fast():
    """The wrappers' host side in C++, for calls with nothing out of the ordinary: each of its
    functions answers None to any other, for the Python code behind it to do or to refuse."""
    global _calls
    if _calls is None:
        import torch
        if not os.path.exists(os.path.join(_HERE, "_torch_calls.so")):
            warnings.warn("_torch_calls.so was not built: small calls take about 10 us longer on the host",
                          RuntimeWarning)
            _calls = _NoCalls
            return _calls
        try:
            from . import _torch_calls
        except ImportError as e:
            raise RuntimeError("_torch_calls.so is of another PyTorch: run %s/build.py (%s)" % (_HERE, e))
        if torch.__version__.split("+")[0] != _torch_calls.torch_version:
            raise RuntimeError("_torch_calls.so was built for PyTorch %s, this is %s: run %s/build.py"
                               % (_torch_calls.torch_version, torch.__version__, _HERE))
        lib = load_library()
        _torch_calls.bind(*(ctypes.cast(getattr(lib, name), _P).value
                            for name in ("attn_rotary", "attn_bwd_workspace_size", "attn_bwd")))
        _calls = _torch_calls
    return _calls


def _bind(torch):
    global _torch, _int32, _float32, _contiguous, _raw_stream, _current_device, _capturing
    _int32, _float32, _contiguous = torch.int32, torch.float32, torch.contiguous_format
    for t in (torch.float32, torch.bfloat16, torch.float16):
        for u in {t, torch.float32}:
            _codes[t, u] = dtype_code(t, u)
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    _capturing = torch._C._cuda_isCurrentStreamCapturing
    _torch = torch  # last: the other names are there for a thread that sees this one


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
    if getattr(stream, "device", device) != device:
        raise ValueError("the tensors are on %s, the stream on %s" % (device, stream.device))
    return stream.cuda_stream


def _on(stream, device):
    """The context in which torch's work and allocations are ``stream``'s, if one is given."""
    if stream is not None and not isinstance(stream, _torch.cuda.Stream):
        stream = _torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return _torch.cuda.stream(stream)


def _new(stream, shape, dtype, device):
    """An uninitialised tensor that belongs to ``stream`` if one is given: memory that the
    current stream's work still uses is then not handed to another stream's."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
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
