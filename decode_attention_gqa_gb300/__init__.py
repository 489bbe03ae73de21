"""GB300 (sm_103a) split-KV grouped-query decode attention.

Thin ctypes binding over ``libattn_decode.so`` (declared in
``include/attn_decode.h``, ``attn_paged.h``, ``attn_tree.h`` and ``attn_pages.h``). Every ``attn_*``
function here has the name and argument order of the C entry point it calls and does argument marshalling only: pointers may
be given as integers or as tensors (their ``data_ptr()`` is passed), streams as
integers, ``torch.cuda.Stream`` objects or ``None`` (the current torch stream).
All arithmetic runs in the library's CUDA kernels; if the library has not been
built, every call raises ``RuntimeError`` -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "AttnError", "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED", "ATTN_ERR_WORKSPACE",
    "ATTN_ERR_CUDA", "ATTN_DEVERR_POSITION_CLAMPED", "ATTN_DEVERR_PIPELINE_TIMEOUT",
    "ATTN_VARIANT_AUTO", "ATTN_VARIANT_SIMT", "ATTN_VARIANT_TC", "ATTN_VARIANT_TCGEN05",
    "ATTN_VARIANT_TCGEN05_CLUSTER", "ATTN_VARIANT_TC_TILE", "ATTN_KV_BF16",
    "ATTN_KV_STABLE",
    "library_path",
    "load",
    "attn_decode", "attn_decode_ex", "attn_decode_append", "attn_decode_multi", "decode_attention",
    "attn_decode_partial",
    "attn_decode_combine",
    "attn_decode_static",
    "attn_split_heuristic", "attn_split_heuristic_ex", "attn_resolve_variant", "attn_plan_call",
    "attn_workspace_size",
    "attn_read_device_error", "attn_selftest_bounded_wait", "attn_status_string",
    "attn_last_cuda_error", "attn_version",
    "ATTN_DEVERR_BAD_PAGE", "ATTN_TYPE_F32", "ATTN_TYPE_F16", "ATTN_TYPE_BF16", "ATTN_TYPE_E4M3",
    "ATTN_ROPE_PLAIN", "ATTN_ROPE_LINEAR", "ATTN_ROPE_BASE", "ATTN_ROPE_BANDS",
    "PagedCache", "Rope", "rope_append", "paged_decode_attention",
    "attn_rope_steps", "attn_rope_append", "attn_decode_paged", "attn_paged_plan",
    "ATTN_DEVERR_BAD_REQUEST", "ATTN_DEVERR_NO_PAGE", "ATTN_DEVERR_SHARED_PAGE",
    "PageBook", "tree_rules", "tree_decode_attention", "keep_rows", "copy_pages",
    "attn_tree_rules", "attn_rope_append_tree", "attn_decode_tree", "attn_tree_plan", "attn_keep_rows",
    "attn_pages_resize", "attn_pages_fork", "attn_pages_copy",
]

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_WORKSPACE, ATTN_ERR_CUDA = range(5)
ATTN_DEVERR_POSITION_CLAMPED = 0x1
ATTN_DEVERR_PIPELINE_TIMEOUT = 0x2
ATTN_VARIANT_AUTO, ATTN_VARIANT_SIMT, ATTN_VARIANT_TC, ATTN_VARIANT_TCGEN05 = 0, 1, 2, 3
ATTN_VARIANT_TCGEN05_CLUSTER = 4
ATTN_VARIANT_TC_TILE = 5
ATTN_KV_BF16 = 0x10
ATTN_KV_STABLE = 0x20
ATTN_DEVERR_BAD_PAGE = 0x4
ATTN_DEVERR_BAD_REQUEST = 0x8
ATTN_DEVERR_NO_PAGE = 0x10
ATTN_DEVERR_SHARED_PAGE = 0x20
ATTN_TYPE_F32, ATTN_TYPE_F16, ATTN_TYPE_BF16, ATTN_TYPE_E4M3 = range(4)
ATTN_ROPE_PLAIN, ATTN_ROPE_LINEAR, ATTN_ROPE_BASE, ATTN_ROPE_BANDS = range(4)

_PKG = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = attn_status_string(status)
        extra = ""
        if status == ATTN_ERR_CUDA:
            extra = " (cudaError %d)" % attn_last_cuda_error()
        super().__init__("%s returned %s%s" % (where, name, extra))


def library_path() -> str:
    return os.path.join(_PKG, "libattn_decode.so")


def load():
    """Load the library (once). Raises RuntimeError if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError("libattn_decode.so is not built (%s); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % path)
        lib = ctypes.CDLL(path)
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.attn_decode.restype = i32
        lib.attn_decode.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp]
        lib.attn_decode_ex.restype = i32
        lib.attn_decode_ex.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i64, i32, i32,
                                       i32, vp, sz, vp]
        lib.attn_decode_append.restype = i32
        lib.attn_decode_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i64,
                                           i32, i32, i32, vp, sz, vp]
        lib.attn_decode_multi.restype = i32
        lib.attn_decode_multi.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i64, i32,
                                          i32, i32, vp, sz, vp]
        lib.attn_decode_partial.restype = i32
        lib.attn_decode_partial.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, f32, i64, i32, i32,
                                            i32, vp, sz, vp]
        lib.attn_decode_combine.restype = i32
        lib.attn_decode_combine.argtypes = [vp, sz, vp, i32, i32, i32, i32, vp]
        lib.attn_decode_static.restype = i32
        lib.attn_decode_static.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i64, i32,
                                           i32, i32, vp]
        lib.attn_split_heuristic.restype = i32
        lib.attn_split_heuristic.argtypes = [i32, i32, i32, i32, i64, i32]
        lib.attn_split_heuristic_ex.restype = i32
        lib.attn_split_heuristic_ex.argtypes = [i32, i32, i32, i32, i32, i64, i32, i32]
        lib.attn_resolve_variant.restype = i32
        lib.attn_resolve_variant.argtypes = [i32, i32, i32, i32, i32, i64, i32, i32]
        lib.attn_plan_call.restype = i32
        lib.attn_plan_call.argtypes = [i32, i32, i32, i32, i32, i64, i32, i32, i32,
                                       ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(sz)]
        lib.attn_workspace_size.restype = sz
        lib.attn_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.attn_read_device_error.restype = i32
        lib.attn_read_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
        lib.attn_selftest_bounded_wait.restype = i32
        lib.attn_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, vp]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_status_string.argtypes = [i32]
        lib.attn_last_cuda_error.restype = i32
        lib.attn_last_cuda_error.argtypes = []
        lib.attn_version.restype = i32
        lib.attn_version.argtypes = []
        f64 = ctypes.c_double
        lib.attn_rope_steps.restype = i32
        lib.attn_rope_steps.argtypes = [i32, f64, i32, f64, f64, f64, i64, vp]
        lib.attn_rope_append.restype = i32
        lib.attn_rope_append.argtypes = [vp, vp, i32, vp, vp, i32, i64, vp, vp, vp, i64, i64, i64,
                                         i32, vp, i32, vp, vp]
        lib.attn_decode_paged.restype = i32
        lib.attn_decode_paged.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, i32, vp,
                                          sz, vp]
        lib.attn_paged_plan.restype = i32
        lib.attn_paged_plan.argtypes = [vp, i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                        ctypes.POINTER(sz)]
        lib.attn_tree_rules.restype = i32
        lib.attn_tree_rules.argtypes = [vp, vp, i32, i64, i32, vp, vp, vp]
        lib.attn_rope_append_tree.restype = i32
        lib.attn_rope_append_tree.argtypes = [vp, vp, i32, vp, vp, i32, i64, vp, vp, vp, i64, i64, i64,
                                              i32, vp, i32, i32, vp, vp, vp]
        lib.attn_decode_tree.restype = i32
        lib.attn_decode_tree.argtypes = [vp, vp, i32, vp, vp, i32, i64, i32, vp, vp, i32, i32, f32, vp,
                                         i32, vp, vp, i32, vp, sz, vp]
        lib.attn_tree_plan.restype = i32
        lib.attn_tree_plan.argtypes = [vp, i32, i32, i64, i32, i32, i32, i32, i32, ctypes.POINTER(i32),
                                       ctypes.POINTER(sz)]
        lib.attn_keep_rows.restype = i32
        lib.attn_keep_rows.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, vp]
        lib.attn_pages_resize.restype = i32
        lib.attn_pages_resize.argtypes = [vp, i32, vp, i32, i32, vp, vp, i32, vp]
        lib.attn_pages_fork.restype = i32
        lib.attn_pages_fork.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp, i32, vp, vp]
        lib.attn_pages_copy.restype = i32
        lib.attn_pages_copy.argtypes = [vp, vp, i32, vp]
        _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    raise TypeError("expected an int address or a tensor, got %r" % type(x))


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    raise TypeError("expected a stream handle, torch.cuda.Stream or None")


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def attn_decode(q, k_cache, v_cache, positions, out, n_seq, n_head, n_kv_head, head_dim, scale,
                stream=None):
    """o = softmax(q·Kᵀ·scale)·V for one sequence (see include/attn_decode.h)."""
    _check(load().attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(positions), _ptr(out),
                              n_seq, n_head, n_kv_head, head_dim, scale, _stream(stream)),
           "attn_decode")


def attn_decode_ex(q, k_cache, v_cache, positions, out, n_seq, n_head, n_kv_head, head_dim, scale,
                   cap, n_splits=0, split_len=0, variant=ATTN_VARIANT_AUTO, workspace=None,
                   workspace_bytes=0, stream=None):
    """Several sequences, explicit capacity, split and workspace control."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    _check(load().attn_decode_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(positions), _ptr(out),
                                 n_seq, n_head, n_kv_head, head_dim, scale, cap, n_splits,
                                 split_len, variant, _ptr(workspace), workspace_bytes,
                                 _stream(stream)),
           "attn_decode_ex")


def decode_attention(q, k_cache, v_cache, positions, scale=None, out=None, n_splits=0,
                     kv_stable=False, stream=None, kernel=ATTN_VARIANT_AUTO):
    """Convenience form of attn_decode_ex for torch tensors: the sizes come
    from the shapes -- q f32 [n_seq, n_head, head_dim] (or [n_seq, n_q,
    n_head, head_dim] for several causal query rows, attn_decode_multi),
    k_cache / v_cache float16 or bfloat16 [n_seq, cap, n_kv_head, head_dim],
    positions int32 [n_seq] -- scale defaults to 1/sqrt(head_dim), the cache
    dtype picks ATTN_KV_BF16, and `out` is allocated when not given. `kernel`
    is one of the ATTN_VARIANT_* values (variant 0, the library's choice, by
    default). The library-owned workspace is used. Returns out."""
    import math
    import torch
    if q.dtype != torch.float32 or positions.dtype != torch.int32:
        raise TypeError("q must be float32 and positions int32")
    if k_cache.dtype != v_cache.dtype or k_cache.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("k_cache and v_cache must both be float16 or both bfloat16")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache / v_cache must be [n_seq, cap, n_kv_head, head_dim]")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("positions", positions)):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    n_seq, cap, n_kv_head, head_dim = k_cache.shape
    if q.dim() == 3:
        n_q, (qs, n_head, qd) = 1, q.shape
    elif q.dim() == 4:
        qs, n_q, n_head, qd = q.shape
    else:
        raise ValueError("q must be [n_seq, n_head, head_dim] or [n_seq, n_q, n_head, head_dim]")
    if qs != n_seq or qd != head_dim or positions.numel() != n_seq:
        raise ValueError("q, the caches and positions disagree on n_seq or head_dim")
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    if out is None:
        out = torch.empty_like(q)
    if kernel not in (ATTN_VARIANT_AUTO, ATTN_VARIANT_SIMT, ATTN_VARIANT_TC, ATTN_VARIANT_TCGEN05,
                      ATTN_VARIANT_TCGEN05_CLUSTER, ATTN_VARIANT_TC_TILE):
        raise ValueError("kernel must be one of the ATTN_VARIANT_* values")
    variant = kernel | (ATTN_KV_BF16 if k_cache.dtype == torch.bfloat16 else 0) | \
        (ATTN_KV_STABLE if kv_stable else 0)
    if n_q > 1:
        attn_decode_multi(q, k_cache, v_cache, positions, out, n_seq, n_q, n_head, n_kv_head,
                          head_dim, scale, cap, n_splits=n_splits, variant=variant, stream=stream)
    else:
        attn_decode_ex(q, k_cache, v_cache, positions, out, n_seq, n_head, n_kv_head, head_dim,
                       scale, cap, n_splits=n_splits, variant=variant, stream=stream)
    return out


def attn_decode_append(q, k_new, v_new, k_cache, v_cache, positions, out, n_seq, n_head, n_kv_head,
                       head_dim, scale, cap, n_splits=0, split_len=0, variant=ATTN_VARIANT_AUTO,
                       workspace=None, workspace_bytes=0, stream=None):
    """Write the new token's K/V row at positions[s] and attend, fused."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    _check(load().attn_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(positions), _ptr(out), n_seq, n_head,
                                     n_kv_head, head_dim, scale, cap, n_splits, split_len, variant,
                                     _ptr(workspace), workspace_bytes, _stream(stream)),
           "attn_decode_append")


def attn_decode_multi(q, k_cache, v_cache, positions, out, n_seq, n_q, n_head, n_kv_head, head_dim,
                      scale, cap, n_splits=0, split_len=0, variant=ATTN_VARIANT_AUTO,
                      workspace=None, workspace_bytes=0, stream=None):
    """n_q causal query rows per sequence (see include/attn_decode.h)."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    _check(load().attn_decode_multi(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(positions),
                                    _ptr(out), n_seq, n_q, n_head, n_kv_head, head_dim, scale, cap,
                                    n_splits, split_len, variant, _ptr(workspace), workspace_bytes,
                                    _stream(stream)),
           "attn_decode_multi")


def attn_decode_partial(q, k_cache, v_cache, positions, n_seq, n_head, n_kv_head, head_dim,
                        scale, cap, n_splits, split_len=0, variant=ATTN_VARIANT_AUTO,
                        workspace=None, workspace_bytes=0, stream=None):
    """Stage one (partials into `workspace`); see include/attn_decode.h."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    _check(load().attn_decode_partial(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(positions),
                                      n_seq, n_head, n_kv_head, head_dim, scale, cap, n_splits,
                                      split_len, variant, _ptr(workspace), workspace_bytes,
                                      _stream(stream)),
           "attn_decode_partial")


def attn_decode_combine(workspace, workspace_bytes, out, n_seq, n_head, head_dim, n_splits,
                        stream=None):
    """Stage two (combine the partials in `workspace` into `out`)."""
    if not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    _check(load().attn_decode_combine(_ptr(workspace), workspace_bytes, _ptr(out), n_seq, n_head,
                                      head_dim, n_splits, _stream(stream)),
           "attn_decode_combine")


def attn_decode_static(q, k_cache, v_cache, positions, out, n_seq, n_head, n_kv_head, head_dim,
                       scale, cap, n_splits=0, split_len=0, variant=ATTN_VARIANT_AUTO, stream=None):
    """attn_decode_ex with the library's fixed scratch array instead of a
    workspace: allocates nothing (see include/attn_decode.h)."""
    _check(load().attn_decode_static(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(positions),
                                     _ptr(out), n_seq, n_head, n_kv_head, head_dim, scale, cap,
                                     n_splits, split_len, variant, _stream(stream)),
           "attn_decode_static")


def attn_split_heuristic(n_seq, n_head, n_kv_head, head_dim, cap, sm_count) -> int:
    return load().attn_split_heuristic(n_seq, n_head, n_kv_head, head_dim, cap, sm_count)


def attn_split_heuristic_ex(n_seq, n_q, n_head, n_kv_head, head_dim, cap, sm_count, variant) -> int:
    return load().attn_split_heuristic_ex(n_seq, n_q, n_head, n_kv_head, head_dim, cap, sm_count,
                                          variant)


def attn_resolve_variant(n_seq, n_q, n_head, n_kv_head, head_dim, cap, sm_count, variant) -> int:
    """The partial kernel (ATTN_VARIANT_SIMT / _TC / _TCGEN05) such a call runs with
    the heuristic's split count; 0 for an unsupported shape."""
    return load().attn_resolve_variant(n_seq, n_q, n_head, n_kv_head, head_dim, cap, sm_count,
                                       variant)


def attn_plan_call(n_seq, n_q, n_head, n_kv_head, head_dim, cap, n_splits=0, split_len=0,
                   variant=0):
    """(kernel variant, split count, workspace bytes) of the call with these
    arguments; raises AttnError with the status the call would return."""
    v = ctypes.c_int(0)
    p = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    _check(load().attn_plan_call(n_seq, n_q, n_head, n_kv_head, head_dim, cap, n_splits, split_len,
                                 variant, ctypes.byref(v), ctypes.byref(p), ctypes.byref(ws)),
           "attn_plan_call")
    return v.value, p.value, ws.value


def attn_workspace_size(n_seq, n_head, head_dim, n_splits) -> int:
    return load().attn_workspace_size(n_seq, n_head, head_dim, n_splits)


def attn_selftest_bounded_wait(limit_ns, stream=None) -> None:
    """Launch the bounded-wait self-test (see include/attn_decode.h)."""
    _check(load().attn_selftest_bounded_wait(limit_ns, _stream(stream)),
           "attn_selftest_bounded_wait")


def attn_read_device_error(stream=None) -> int:
    flags = ctypes.c_uint(0)
    _check(load().attn_read_device_error(_stream(stream), ctypes.byref(flags)),
           "attn_read_device_error")
    return flags.value


def attn_status_string(status) -> str:
    return load().attn_status_string(status).decode()


def attn_last_cuda_error() -> int:
    return load().attn_last_cuda_error()


def attn_version() -> int:
    return load().attn_version()


# ---------------------------------------------------------------------------
# Paged cache (include/attn_paged.h).
# ---------------------------------------------------------------------------
class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_head", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class _RulesStruct(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("starts", ctypes.c_void_p)]


def attn_rope_steps(rot_dim, base, scaling=ATTN_ROPE_PLAIN, factor=1.0, low_turns=0.0,
                    high_turns=0.0, trained_len=0):
    """The rotary steps per position as a list of rot_dim / 2 integers below 2^64 (host-only)."""
    out = (ctypes.c_uint64 * max(1, min(int(rot_dim), 256) // 2))()
    _check(load().attn_rope_steps(rot_dim, base, scaling, factor, low_turns, high_turns,
                                  trained_len, ctypes.addressof(out)), "attn_rope_steps")
    return list(out)


def attn_rope_append(cache, block_table, max_pages, positions, cu_tokens, n_seq, n_tokens, q, k_new,
                     v_new, q_stride, k_stride, v_stride, in_type, q_out, n_head, rope=None,
                     stream=None):
    """Rotate q and k by position and write k, v into the paged cache. `cache` and `rope` are a
    PagedCache and a Rope (or addresses of the C structures)."""
    _check(load().attn_rope_append(_struct(cache), _ptr(block_table), max_pages, _ptr(positions),
                                   _ptr(cu_tokens), n_seq, n_tokens, _ptr(q), _ptr(k_new),
                                   _ptr(v_new), q_stride, k_stride, v_stride, in_type, _ptr(q_out),
                                   n_head, _struct(rope), _stream(stream)),
           "attn_rope_append")


def attn_paged_plan(cache, max_pages, n_seq, n_q, n_head, window=0, n_splits=0, sm_count=0):
    """(split count, workspace bytes) of the attn_decode_paged call with these arguments."""
    p, ws = ctypes.c_int(0), ctypes.c_size_t(0)
    _check(load().attn_paged_plan(_struct(cache), max_pages, n_seq, n_q, n_head, window, n_splits,
                                  sm_count, ctypes.byref(p), ctypes.byref(ws)), "attn_paged_plan")
    return p.value, ws.value


def attn_decode_paged(cache, block_table, max_pages, positions, q, out, n_seq, n_q, n_head, scale,
                      rules=None, n_splits=0, workspace=None, workspace_bytes=0, stream=None):
    """Decode attention over the paged cache. `rules` is None or the (softcap, window, slopes,
    starts) of attn_score_rules."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    if rules is not None:
        softcap, window, slopes, starts = rules
        rules = _rules(softcap, window, _ptr(slopes), _ptr(starts))
        rules_p = ctypes.addressof(rules)
    else:
        rules_p = None
    _check(load().attn_decode_paged(_struct(cache), _ptr(block_table), max_pages, _ptr(positions),
                                    _ptr(q), _ptr(out), n_seq, n_q, n_head, scale, rules_p,
                                    n_splits, _ptr(workspace), workspace_bytes, _stream(stream)),
           "attn_decode_paged")


def attn_tree_rules(parents, cu_tokens, n_seq, n_tokens, max_nodes, mask, depths, stream=None):
    """Masks and depths of the nodes of trees from their parents."""
    _check(load().attn_tree_rules(_ptr(parents), _ptr(cu_tokens), n_seq, n_tokens, max_nodes, _ptr(mask),
                                  _ptr(depths), _stream(stream)), "attn_tree_rules")


def attn_rope_append_tree(cache, block_table, max_pages, positions, cu_tokens, n_seq, n_tokens, q, k_new,
                          v_new, q_stride, k_stride, v_stride, in_type, q_out, out_type, n_head, rope=None,
                          depths=None, stream=None):
    """attn_rope_append with angles by depth and q_out of out_type."""
    _check(load().attn_rope_append_tree(_struct(cache), _ptr(block_table), max_pages, _ptr(positions),
                                        _ptr(cu_tokens), n_seq, n_tokens, _ptr(q), _ptr(k_new), _ptr(v_new),
                                        q_stride, k_stride, v_stride, in_type, _ptr(q_out), out_type, n_head,
                                        _struct(rope), _ptr(depths), _stream(stream)),
           "attn_rope_append_tree")


def attn_tree_plan(cache, max_pages, n_seq, n_tokens, max_nodes, q_type, n_head, n_splits=0, sm_count=0):
    """(split count, workspace bytes) of the attn_decode_tree call with these arguments."""
    p, ws = ctypes.c_int(0), ctypes.c_size_t(0)
    _check(load().attn_tree_plan(_struct(cache), max_pages, n_seq, n_tokens, max_nodes, q_type, n_head,
                                 n_splits, sm_count, ctypes.byref(p), ctypes.byref(ws)), "attn_tree_plan")
    return p.value, ws.value


def attn_decode_tree(cache, block_table, max_pages, positions, cu_tokens, n_seq, n_tokens, max_nodes, q, out,
                     q_type, n_head, scale, mask=None, mask_words=0, depths=None, rules=None, n_splits=0,
                     workspace=None, workspace_bytes=0, stream=None):
    """Attention of the nodes of trees. `rules` is None or the (softcap, window, slopes, starts) of
    attn_score_rules."""
    if workspace is not None and not workspace_bytes and hasattr(workspace, "nbytes"):
        workspace_bytes = workspace.nbytes
    rules_p = None
    if rules is not None:
        softcap, window, slopes, starts = rules
        rules = _rules(softcap, window, _ptr(slopes), _ptr(starts))
        rules_p = ctypes.addressof(rules)
    _check(load().attn_decode_tree(_struct(cache), _ptr(block_table), max_pages, _ptr(positions),
                                   _ptr(cu_tokens), n_seq, n_tokens, max_nodes, _ptr(q), _ptr(out), q_type,
                                   n_head, scale, _ptr(mask), mask_words, _ptr(depths), rules_p, n_splits,
                                   _ptr(workspace), workspace_bytes, _stream(stream)), "attn_decode_tree")


def attn_keep_rows(cache, block_table, max_pages, base, path, counts, n_seq, max_keep, stream=None):
    """Move the kept rows behind base together."""
    _check(load().attn_keep_rows(_struct(cache), _ptr(block_table), max_pages, _ptr(base), _ptr(path),
                                 _ptr(counts), n_seq, max_keep, _stream(stream)), "attn_keep_rows")


def attn_pages_resize(refs, n_pages, block_table, max_pages, page_size, have, want, n_seq, stream=None):
    """Release and give out pages, from have to want rows."""
    _check(load().attn_pages_resize(_ptr(refs), n_pages, _ptr(block_table), max_pages, page_size, _ptr(have),
                                    _ptr(want), n_seq, _stream(stream)), "attn_pages_resize")


def attn_pages_fork(refs, n_pages, block_table, max_pages, page_size, n_seq, src, dst, rows, n_fork, copies,
                    stream=None):
    """Share the pages of src with dst; what is left to copy goes to copies."""
    _check(load().attn_pages_fork(_ptr(refs), n_pages, _ptr(block_table), max_pages, page_size, n_seq,
                                  _ptr(src), _ptr(dst), _ptr(rows), n_fork, _ptr(copies), _stream(stream)),
           "attn_pages_fork")


def attn_pages_copy(cache, copies, n, stream=None):
    """Copy rows of pages to other pages."""
    _check(load().attn_pages_copy(_struct(cache), _ptr(copies), n, _stream(stream)), "attn_pages_copy")


def _rules(softcap, window, slopes, starts):
    r = _RulesStruct(softcap, window, slopes, starts)
    if softcap and not r.softcap:
        raise ValueError("softcap is 0 in 32 bits, which stands for none")
    return r


def _struct(x):
    if x is None or isinstance(x, int):
        return x
    return x._address


# The torch forms below check their tensors in one expression, since a decode step's call costs the host
# more than the GPU; `_refuse` finds out what was wrong with them.
_torch = None


def _torch_module():
    global _torch, _alloc, _free, _device, _raw_stream
    if _torch is None:
        import torch
        # torch's allocator without a tensor around the memory, the current device, and a stream's handle without an
        # object; by their public names where these are missing
        c = torch._C
        _alloc = getattr(c, "_cuda_cudaCachingAllocator_raw_alloc", None)
        _free = getattr(c, "_cuda_cudaCachingAllocator_raw_delete", None)
        if _alloc is None or _free is None:
            def _alloc(size, stream):
                return torch.cuda.caching_allocator_alloc(size, stream=stream)
            _free = torch.cuda.caching_allocator_delete
        _device = getattr(c, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(c, "_cuda_getCurrentRawStream", None)
        if _raw_stream is None:
            def _raw_stream(index):
                return torch.cuda.current_stream(index).cuda_stream
        _torch = torch
    return _torch


def _on_device(name, t, dtype, device):
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, str(dtype).replace("torch.", "")))
    if t.device != device:
        raise ValueError("%s must be on %s, the cache's device" % (name, device))


def _dense(name, t):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _refuse(checks, device, shapes):
    """Raise for the first of `checks` (name, tensor, dtype, dense) or of `shapes` (holds, message)
    that fails."""
    _same_device(device)
    for name, t, dtype, dense in checks:
        if t is not None:
            _on_device(name, t, dtype, device)
            if dense:
                _dense(name, t)
    for holds, message in shapes:
        if not holds:
            raise ValueError(message)
    raise ValueError("the tensors do not fit together")


class PagedCache:
    """The pool of a paged cache: k, v [n_pages, page_size, n_kv_head, head_dim] float16, bfloat16
    or float8_e4m3fn, as torch tensors of any strides over the first three dimensions (the same for
    both, at least head_dim; the last one dense); k_scale, v_scale float32 [n_pages, n_kv_head] for float8_e4m3fn.
    Holds the tensors and the C structure that describes them."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        types = {torch.float16: ATTN_TYPE_F16, torch.bfloat16: ATTN_TYPE_BF16,
                 torch.float8_e4m3fn: ATTN_TYPE_E4M3}
        if k.dtype not in types or v.dtype != k.dtype:
            raise TypeError("k and v must both be float16, bfloat16 or float8_e4m3fn")
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [n_pages, page_size, n_kv_head, head_dim]")
        # a dimension of one element has no stride
        strides, vstrides = ([t.stride(i) if t.shape[i] > 1 else t.shape[3] for i in range(3)] for t in (k, v))
        if strides != vstrides or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must have the same strides, and dense rows")
        if min(strides) < k.shape[3]:        # three strides of 0 would stand for a dense pool
            raise ValueError("rows of k and v must not overlap (strides below head_dim)")
        if v.device != k.device:
            raise ValueError("k and v must be on the same device")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache, and it needs both")
        n_pages, page_size, n_kv_head, head_dim = k.shape
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _on_device(name, t, torch.float32, k.device)
                if t.shape != (n_pages, n_kv_head):
                    raise ValueError("%s must be [n_pages, n_kv_head]" % name)
                _dense(name, t)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_kv_head, self.head_dim, self.page_size = n_kv_head, head_dim, page_size
        self.device = k.device
        self._c = _CacheStruct(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                               *strides, n_pages, page_size, n_kv_head,
                               head_dim, types[k.dtype], 0)
        self._address = ctypes.addressof(self._c)
        self._index = k.get_device()
        self._plans = {}


class Rope:
    """The rotation of rope_append: rotary steps on the device, made by attn_rope_steps, with the
    rotated dimensions, the layout and the magnitude of attn_rope."""

    def __init__(self, rot_dim, base=10000.0, scaling=ATTN_ROPE_PLAIN, factor=1.0, low_turns=0.0,
                 high_turns=0.0, trained_len=0, interleaved=False, mscale=1.0, device="cuda"):
        import torch
        steps = attn_rope_steps(rot_dim, base, scaling, factor, low_turns, high_turns, trained_len)
        self.steps = torch.tensor([s - (1 << 64) if s >> 63 else s for s in steps],
                                  dtype=torch.int64, device=device)
        self.rot_dim = rot_dim
        self._index = self.steps.get_device()
        self._c = _RopeStruct(self.steps.data_ptr(), rot_dim, 1 if interleaved else 0, mscale, 0)
        self._address = ctypes.addressof(self._c)


def _same_device(device):
    if device.type != "cuda" or device.index != _torch_module().cuda.current_device():
        raise ValueError("the cache must be on the current CUDA device")


def _in_type(dtype, name="k_new"):
    torch = _torch_module()
    if dtype is torch.bfloat16:
        return ATTN_TYPE_BF16
    if dtype is torch.float16:
        return ATTN_TYPE_F16
    if dtype is torch.float32:
        return ATTN_TYPE_F32
    raise TypeError("%s must be float32, float16 or bfloat16" % name)


def rope_append(cache, block_table, positions, k_new, v_new, q=None, q_out=None, rope=None,
                cu_tokens=None, stream=None, depths=None):
    """Convenience form of attn_rope_append for torch tensors: the sizes come from the shapes --
    k_new, v_new [n_tokens, n_kv_head, head_dim] and q [n_tokens, n_head, head_dim] (or None) of one
    type (float32, float16 or bfloat16), dense within a token and of any stride between tokens that
    do not overlap (a row repeated by expand is refused; pass its contiguous() copy);
    block_table int32 [n_seq, max_pages]; positions int32 [n_seq]; cu_tokens int32 [n_seq + 1], or
    None for the same number of tokens in every sequence; depths int32 [n_tokens] for the nodes of
    trees (attn_rope_append_tree), or None. `q_out` (float32, or the type of q) is allocated as float32
    when not given (on the current stream, so another `stream` needs it given). Returns q_out (None
    without q)."""
    torch = _torch or _torch_module()
    i32, index, dt, hd = torch.int32, cache._index, k_new.dtype, cache.head_dim
    in_type = _in_type(dt)
    shape, ks, vs = k_new.shape, k_new.stride(), v_new.stride()
    n_tokens, n_kv = shape[0], cache.n_kv_head
    n_seq, max_pages = block_table.shape if block_table.dim() == 2 else (-1, 0)
    row = (n_kv, hd)
    if not (index >= 0 and index == _device() and shape[1:] == row and v_new.shape == shape and
            v_new.dtype is dt and k_new.get_device() == index and v_new.get_device() == index and
            ks[2] == 1 and vs[2] == 1 and (n_kv == 1 or (ks[1] == hd and vs[1] == hd)) and
            block_table.dtype is i32 and block_table.get_device() == index and block_table.is_contiguous() and
            positions.dtype is i32 and positions.get_device() == index and positions.is_contiguous() and
            positions.shape == (n_seq,)):
        _refuse((("k_new", k_new, dt, False), ("v_new", v_new, dt, False),
                 ("block_table", block_table, i32, True), ("positions", positions, i32, True)), cache.device,
                ((shape[1:] == row and v_new.shape == shape, "k_new and v_new must be [n_tokens, n_kv_head, head_dim]"),
                 (n_seq >= 0 and positions.shape == (n_seq,),
                  "block_table must be [n_seq, max_pages] and positions [n_seq]"),
                 (False, "k_new and v_new must be dense within a token")))
    qs = n_head = 0
    out_type = ATTN_TYPE_F32
    qp = op = cp = dp = None
    if q is not None:
        qshape, qst = q.shape, q.stride()
        if not (len(qshape) == 3 and qshape[0] == n_tokens and qshape[2] == hd and q.dtype is dt and
                q.get_device() == index and qst[2] == 1 and (qshape[1] == 1 or qst[1] == hd)):
            _refuse((("q", q, dt, False),), cache.device,
                    ((False, "q must be [n_tokens, n_head, head_dim], dense within a token"),))
        n_head, qs = qshape[1], qst[0]
        if q_out is None:
            if stream is not None and _stream(stream) != _raw_stream(index):
                raise ValueError("q_out must be given with a stream that is not the current one")
            q_out = torch.empty(qshape, dtype=torch.float32, device=cache.device)
        elif not (q_out.shape == qshape and q_out.dtype in (torch.float32, dt) and q_out.get_device() == index and
                  q_out.is_contiguous()):
            _refuse((("q_out", q_out, dt if q_out.dtype is dt else torch.float32, True),), cache.device,
                    ((False, "q_out must have the shape of q"),))
        if q_out.dtype is not torch.float32:
            out_type = in_type
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if cu_tokens is not None:
        if not (cu_tokens.dtype is i32 and cu_tokens.get_device() == index and cu_tokens.shape == (n_seq + 1,) and
                cu_tokens.is_contiguous()):
            _refuse((("cu_tokens", cu_tokens, i32, True),), cache.device,
                    ((False, "cu_tokens must be [n_seq + 1]"),))
        cp = cu_tokens.data_ptr()
    if depths is not None:
        if not (depths.dtype is i32 and depths.get_device() == index and depths.shape == (n_tokens,) and
                depths.is_contiguous()):
            _refuse((("depths", depths, i32, True),), cache.device, ((False, "depths must be [n_tokens]"),))
        dp = depths.data_ptr()
    rp = None
    if rope is not None:
        if rope._index != index:
            raise ValueError("rope must be on the cache's device")
        rp = rope._address
    if n_tokens <= 1:
        qs, kst, vst = 0, 0, 0                       # one token has no stride
    else:
        # the C call takes a stride of 0 for dense, and would read past the end of a row repeated by expand
        kst, vst = ks[0], vs[0]
        if kst < n_kv * hd or vst < n_kv * hd or qs < n_head * hd:
            _refuse((), cache.device, [(st >= h * hd, "%s must not have tokens that overlap" % name) for name, st, h in
                                       (("k_new", kst, n_kv), ("v_new", vst, n_kv), ("q", qs, n_head))])
    status = (_lib or load()).attn_rope_append_tree(
        cache._address, block_table.data_ptr(), max_pages, positions.data_ptr(), cp, n_seq, n_tokens, qp,
        k_new.data_ptr(), v_new.data_ptr(), qs, kst, vst, in_type, op, out_type, n_head, rp, dp,
        _raw_stream(index) if stream is None else _stream(stream))
    if status:
        raise AttnError(status, "attn_rope_append")
    return q_out


def paged_decode_attention(cache, block_table, positions, q, scale=None, out=None, softcap=0.0,
                           slopes=None, window=0, starts=None, n_splits=0, stream=None):
    """Convenience form of attn_decode_paged for torch tensors: q float32 [n_seq, n_head, head_dim],
    or [n_seq, n_q, n_head, head_dim] for several causal query rows; block_table int32 [n_seq,
    max_pages]; positions int32 [n_seq]; slopes float32 [n_head] and starts int32 [n_seq] or None.
    scale defaults to 1/sqrt(head_dim) and `out` is allocated when not given. The workspace comes
    from torch's allocator on the current stream (pass that stream, or None: another one would
    not be ordered with the workspace's reuse), so captured graphs hold workspaces of their own.
    Returns out."""
    torch = _torch or _torch_module()
    i32, f32, index, hd = torch.int32, torch.float32, cache._index, cache.head_dim
    shape = q.shape
    if len(shape) == 3:
        n_q, (qs, n_head, qd) = 1, shape
    elif len(shape) == 4:
        qs, n_q, n_head, qd = shape
    else:
        raise ValueError("q must be [n_seq, n_head, head_dim] or [n_seq, n_q, n_head, head_dim]")
    n_seq, max_pages = block_table.shape if block_table.dim() == 2 else (-1, 0)
    if not (index >= 0 and index == _device() and qs == n_seq and qd == hd and q.dtype is f32 and
            q.get_device() == index and q.is_contiguous() and
            block_table.dtype is i32 and block_table.get_device() == index and block_table.is_contiguous() and
            positions.dtype is i32 and positions.get_device() == index and positions.is_contiguous() and
            positions.shape == (n_seq,)):
        _refuse((("block_table", block_table, i32, True), ("positions", positions, i32, True), ("q", q, f32, True)),
                cache.device,
                ((n_seq >= 0 and positions.shape == (n_seq,),
                  "block_table must be [n_seq, max_pages] and positions [n_seq]"),
                 (False, "q, the cache and positions disagree on n_seq or head_dim")))
    if out is None:
        out = torch.empty_like(q)
    elif not (out.shape == shape and out.dtype is f32 and out.get_device() == index and out.is_contiguous()):
        _refuse((("out", out, f32, True),), cache.device, ((False, "out must have the shape of q"),))
    rules = None
    if softcap or window or slopes is not None or starts is not None:
        if slopes is not None and not (slopes.dtype is f32 and slopes.get_device() == index and
                                       slopes.shape == (n_head,) and slopes.is_contiguous()):
            _refuse((("slopes", slopes, f32, True),), cache.device, ((False, "slopes must be [n_head]"),))
        if starts is not None and not (starts.dtype is i32 and starts.get_device() == index and
                                       starts.shape == (n_seq,) and starts.is_contiguous()):
            _refuse((("starts", starts, i32, True),), cache.device, ((False, "starts must be [n_seq]"),))
        kept = _rules(softcap, window, slopes.data_ptr() if slopes is not None else None,
                      starts.data_ptr() if starts is not None else None)
        rules = ctypes.addressof(kept)
    if n_seq == 0:
        return out
    handle = _raw_stream(index)
    if stream is not None and _stream(stream) != handle:
        raise ValueError("stream must be the current stream (torch.cuda.stream selects one)")
    # the plan is a function of these numbers, the pool's shape and the device
    key = (max_pages, n_seq, n_q, n_head, window, n_splits)
    plan = cache._plans.get(key)
    if plan is None:
        if not (0 <= window < 1 << 31 and 0 <= n_splits < 1 << 31):
            raise ValueError("window and n_splits must be non-negative 32-bit integers")
        if len(cache._plans) >= 4096:
            cache._plans.clear()
        plan = cache._plans[key] = attn_paged_plan(cache, max_pages, n_seq, n_q, n_head, window, n_splits)
    n_splits, need = plan
    ws = _alloc(need, handle) if need else None
    try:
        status = (_lib or load()).attn_decode_paged(
            cache._address, block_table.data_ptr(), max_pages, positions.data_ptr(), q.data_ptr(), out.data_ptr(),
            n_seq, n_q, n_head, hd ** -0.5 if scale is None else scale, rules, n_splits, ws, need, handle)
    finally:
        if need:
            _free(ws)                   # for what follows on this stream
    if status:
        raise AttnError(status, "attn_decode_paged")
    return out


# ---------------------------------------------------------------------------
# Drafted trees (include/attn_tree.h) and page bookkeeping (include/attn_pages.h).
# ---------------------------------------------------------------------------
def _ints(name, t, shape, index, device):
    """The address of an int32 tensor of this shape on the device (None: None)."""
    if t is None:
        return None
    if not (t.dtype is _torch.int32 and t.get_device() == index and t.shape == shape and t.is_contiguous()):
        _refuse(((name, t, _torch.int32, True),), device,
                ((False, "%s must be [%s]" % (name, ", ".join(str(n) for n in shape))),))
    return t.data_ptr()


def _current(t):
    """The index of the current device, which `t` must be on."""
    index = t.get_device()
    if index < 0 or index != _device():
        raise ValueError("the tensors must be on the current CUDA device")
    return index


def _nodes_of(cu_tokens, n_tokens, n_seq, max_nodes):
    if cu_tokens is None:
        if n_seq < 1 or n_tokens % n_seq:
            raise ValueError("without cu_tokens every sequence has the same number of nodes")
        return max(n_tokens // n_seq, 1) if max_nodes is None else max_nodes
    if max_nodes is None:
        raise ValueError("max_nodes belongs to cu_tokens")
    return max_nodes


def tree_rules(parents, cu_tokens=None, max_nodes=None, mask=None, depths=None, stream=None):
    """Convenience form of attn_tree_rules for torch tensors: parents int32 [n_seq, n] (n nodes in every
    sequence), or [n_tokens] with cu_tokens int32 [n_seq + 1] and max_nodes, which bounds the nodes of a
    sequence. Returns (mask int32 [n_tokens, (max_nodes + 31) // 32], depths int32 [n_tokens]), allocated
    when not given (on the current stream, so another `stream` needs them given)."""
    torch = _torch or _torch_module()
    index = _current(parents)
    device, i32 = parents.device, torch.int32
    if cu_tokens is None:
        if parents.dim() != 2:
            raise ValueError("parents must be [n_seq, n], or [n_tokens] with cu_tokens")
        n_seq = parents.shape[0]
        n_tokens = parents.numel()
    else:
        if parents.dim() != 1 or cu_tokens.dim() != 1 or cu_tokens.shape[0] < 1:
            raise ValueError("parents must be [n_tokens] and cu_tokens [n_seq + 1]")
        n_seq, n_tokens = cu_tokens.shape[0] - 1, parents.shape[0]
    if cu_tokens is not None or n_seq:
        max_nodes = _nodes_of(cu_tokens, n_tokens, n_seq, max_nodes)
    else:
        max_nodes = 1 if max_nodes is None else max_nodes
    if stream is not None and (mask is None or depths is None) and _stream(stream) != _raw_stream(index):
        raise ValueError("mask and depths must be given with a stream that is not the current one")
    words = (max_nodes + 31) // 32
    if mask is None:
        mask = torch.empty((n_tokens, words), dtype=i32, device=device)
    if depths is None:
        depths = torch.empty(n_tokens, dtype=i32, device=device)
    status = (_lib or load()).attn_tree_rules(
        _ints("parents", parents, parents.shape, index, device),
        _ints("cu_tokens", cu_tokens, (n_seq + 1,), index, device), n_seq, n_tokens, max_nodes,
        _ints("mask", mask, (n_tokens, words), index, device), _ints("depths", depths, (n_tokens,), index, device),
        _raw_stream(index) if stream is None else _stream(stream))
    if status:
        raise AttnError(status, "attn_tree_rules")
    return mask, depths


def tree_decode_attention(cache, block_table, positions, q, mask=None, depths=None, cu_tokens=None, max_nodes=None,
                          scale=None, out=None, softcap=0.0, slopes=None, window=0, starts=None, n_splits=0,
                          stream=None):
    """Convenience form of attn_decode_tree for torch tensors: q float32, float16 or bfloat16
    [n_tokens, n_head, head_dim], or [n_seq, n, n_head, head_dim] for n nodes in every sequence; mask int32
    [n_tokens, words] and depths int32 [n_tokens] as tree_rules gives them, or None for chains; cu_tokens int32
    [n_seq + 1] with max_nodes where sequences have different numbers of nodes; the rest as in
    paged_decode_attention. Returns out, of the shape and type of q."""
    torch = _torch or _torch_module()
    i32, f32, index, hd, device = torch.int32, torch.float32, cache._index, cache.head_dim, cache.device
    shape = q.shape
    n_seq, max_pages = block_table.shape if block_table.dim() == 2 else (-1, 0)
    if len(shape) == 3:
        n_tokens, n_head, qd = shape
    elif len(shape) == 4 and cu_tokens is None:
        n_tokens, n_head, qd = shape[0] * shape[1], shape[2], shape[3]
        if shape[0] != n_seq:
            n_seq = -1
    else:
        raise ValueError("q must be [n_tokens, n_head, head_dim], or [n_seq, n, n_head, head_dim] without cu_tokens")
    q_type = _in_type(q.dtype, "q")
    if not (index >= 0 and index == _device() and n_seq >= 0 and qd == hd and q.get_device() == index and
            q.is_contiguous() and
            block_table.dtype is i32 and block_table.get_device() == index and block_table.is_contiguous() and
            positions.dtype is i32 and positions.get_device() == index and positions.is_contiguous() and
            positions.shape == (n_seq,)):
        _refuse((("block_table", block_table, i32, True), ("positions", positions, i32, True),
                 ("q", q, q.dtype, True)), device,
                ((n_seq >= 0 and positions.shape == (n_seq,),
                  "block_table must be [n_seq, max_pages], positions [n_seq] and q of as many sequences"),
                 (False, "q and the cache disagree on head_dim")))
    if out is None:
        out = torch.empty_like(q)
    elif not (out.shape == shape and out.dtype is q.dtype and out.get_device() == index and out.is_contiguous()):
        _refuse((("out", out, q.dtype, True),), device, ((False, "out must have the shape of q"),))
    if n_seq == 0 and n_tokens == 0:
        return out
    max_nodes = _nodes_of(cu_tokens, n_tokens, n_seq, max_nodes)
    words = 0
    if mask is not None:
        words = mask.shape[1] if mask.dim() == 2 else -1
        if words < (max_nodes + 31) // 32:                # none has no address, which stands for chains
            raise ValueError("mask must be [n_tokens, words] with a bit for each of max_nodes nodes")
        mask = _ints("mask", mask, (n_tokens, words), index, device)
    rules = None
    if softcap or window or slopes is not None or starts is not None:
        if not 0 <= window < 1 << 31:                     # the plan does not know it
            raise ValueError("window must be a non-negative 32-bit integer")
        if slopes is not None and not (slopes.dtype is f32 and slopes.get_device() == index and
                                       slopes.shape == (n_head,) and slopes.is_contiguous()):
            _refuse((("slopes", slopes, f32, True),), device, ((False, "slopes must be [n_head]"),))
        kept = _rules(softcap, window, slopes.data_ptr() if slopes is not None else None,
                      _ints("starts", starts, (n_seq,), index, device))
        rules = ctypes.addressof(kept)
    if n_tokens == 0:
        return out
    handle = _raw_stream(index)
    if stream is not None and _stream(stream) != handle:
        raise ValueError("stream must be the current stream (torch.cuda.stream selects one)")
    key = (max_pages, n_seq, n_tokens, max_nodes, q_type, n_head, n_splits, "tree")
    plan = cache._plans.get(key)
    if plan is None:
        if not (0 <= n_splits < 1 << 31 and 0 < max_nodes < 1 << 31):
            raise ValueError("n_splits and max_nodes must be non-negative 32-bit integers")
        if len(cache._plans) >= 4096:
            cache._plans.clear()
        plan = cache._plans[key] = attn_tree_plan(cache, max_pages, n_seq, n_tokens, max_nodes, q_type, n_head,
                                                  n_splits)
    n_splits, need = plan
    ws = _alloc(need, handle) if need else None
    try:
        status = (_lib or load()).attn_decode_tree(
            cache._address, block_table.data_ptr(), max_pages, positions.data_ptr(),
            _ints("cu_tokens", cu_tokens, (n_seq + 1,), index, device), n_seq, n_tokens, max_nodes, q.data_ptr(),
            out.data_ptr(), q_type, n_head, hd ** -0.5 if scale is None else scale, mask, words,
            _ints("depths", depths, (n_tokens,), index, device), rules, n_splits, ws, need, handle)
    finally:
        if need:
            _free(ws)                   # for what follows on this stream
    if status:
        raise AttnError(status, "attn_decode_tree")
    return out


def keep_rows(cache, block_table, base, path, counts, stream=None):
    """Convenience form of attn_keep_rows for torch tensors: row base[s] + path[s, i] of sequence s becomes row
    base[s] + i for i < counts[s]; block_table int32 [n_seq, max_pages], base and counts int32 [n_seq], path
    int32 [n_seq, max_keep]."""
    _torch or _torch_module()
    index, device = cache._index, cache.device
    if index < 0 or index != _device():
        _same_device(device)
    if block_table.dim() != 2 or path.dim() != 2:
        raise ValueError("block_table must be [n_seq, max_pages] and path [n_seq, max_keep]")
    n_seq, max_keep = path.shape
    max_pages = block_table.shape[1]
    status = (_lib or load()).attn_keep_rows(
        cache._address, _ints("block_table", block_table, (n_seq, max_pages), index, device), max_pages,
        _ints("base", base, (n_seq,), index, device), _ints("path", path, (n_seq, max_keep), index, device),
        _ints("counts", counts, (n_seq,), index, device), n_seq, max_keep,
        _raw_stream(index) if stream is None else _stream(stream))
    if status:
        raise AttnError(status, "attn_keep_rows")


def copy_pages(cache, copies, stream=None):
    """Convenience form of attn_pages_copy for torch tensors: copies int32 [n, 4], as PageBook.fork gives them."""
    _torch or _torch_module()
    index, device = cache._index, cache.device
    if index < 0 or index != _device():
        _same_device(device)
    n = copies.shape[0] if copies.dim() == 2 else -1
    status = (_lib or load()).attn_pages_copy(cache._address, _ints("copies", copies, (n, 4), index, device), n,
                                              _raw_stream(index) if stream is None else _stream(stream))
    if status:
        raise AttnError(status, "attn_pages_copy")


class PageBook:
    """The pages of a paged cache (or of the caches of all layers, where they use the same numbers): refs int32
    [n_pages], how many block-table entries hold each page, and the block table int32 [n_seq, max_pages]. Holds
    the tensors; its calls change them in place, on the device (include/attn_pages.h)."""

    def __init__(self, refs, block_table, page_size):
        torch = _torch_module()
        if refs.device != block_table.device or refs.get_device() < 0:
            raise ValueError("refs and block_table must be on the same CUDA device")
        for name, t, dims in (("refs", refs, 1), ("block_table", block_table, 2)):
            _on_device(name, t, torch.int32, refs.device)
            _dense(name, t)
            if t.dim() != dims:
                raise ValueError("refs must be [n_pages] and block_table [n_seq, max_pages]")
        self.refs, self.block_table, self.page_size = refs, block_table, page_size
        self._index, self.device = refs.get_device(), refs.device

    def _at(self, stream):
        if self._index != _device():
            raise ValueError("refs and block_table must be on the current CUDA device")
        return _raw_stream(self._index) if stream is None else _stream(stream)

    def resize(self, have, want, stream=None):
        """attn_pages_resize: every sequence from have to want rows (int32 [n_seq])."""
        handle = self._at(stream)
        n_seq, max_pages = self.block_table.shape
        status = (_lib or load()).attn_pages_resize(
            self.refs.data_ptr(), self.refs.shape[0], self.block_table.data_ptr(), max_pages, self.page_size,
            _ints("have", have, (n_seq,), self._index, self.device),
            _ints("want", want, (n_seq,), self._index, self.device), n_seq, handle)
        if status:
            raise AttnError(status, "attn_pages_resize")

    def fork(self, src, dst, rows, copies=None, stream=None):
        """attn_pages_fork: sequence dst[i] takes the first rows[i] rows of src[i] (int32 [n_fork]). Returns
        copies int32 [n_fork, 4] for copy_pages, allocated when not given (on the current stream, so another
        `stream` needs it given)."""
        handle = self._at(stream)
        n = src.shape[0] if src.dim() == 1 else -1
        if copies is None:
            if stream is not None and handle != _raw_stream(self._index):
                raise ValueError("copies must be given with a stream that is not the current one")
            copies = _torch.empty((max(n, 0), 4), dtype=_torch.int32, device=self.device)
        n_seq, max_pages = self.block_table.shape
        status = (_lib or load()).attn_pages_fork(
            self.refs.data_ptr(), self.refs.shape[0], self.block_table.data_ptr(), max_pages, self.page_size, n_seq,
            _ints("src", src, (n,), self._index, self.device), _ints("dst", dst, (n,), self._index, self.device),
            _ints("rows", rows, (n,), self._index, self.device), n,
            _ints("copies", copies, (n, 4), self._index, self.device), handle)
        if status:
            raise AttnError(status, "attn_pages_fork")
        return copies
