"""Python binding of the R-SWA C ABI (librswa.so).

Argument marshalling only: every entry point converts torch tensors to device
pointers and calls the function of the same name in the shared library, which
does all of the work in CUDA kernels.  There is no Python or CPU fallback: if
the library is missing, ``load()`` raises.

Layouts (see include/rswa.h): prefill tensors are token-major packed rows
``[sum_b (m_b + T)][H][d]``; per-step tensors are ``[B][H][d]``; ``lse`` is
``[B][H]`` float32.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "RswaError", "load", "library_path", "declared_symbols",
    "RSWA_F32", "RSWA_BF16",
    "rswa_strerror", "rswa_cache_footprint", "rswa_cache_create",
    "rswa_cache_footprint_gqa", "rswa_cache_create_gqa", "rswa_prefill_varlen",
    "rswa_cache_destroy", "rswa_prefill", "rswa_append_kv",
    "rswa_decode_step", "rswa_decode_step_fused",
    "rswa_decode_step_fused_static", "rswa_decode_block", "rswa_cache_bytes",
    "rswa_cache_len", "rswa_cache_get_t", "rswa_cache_set_t",
    "rswa_sync_status", "rswa_debug_fail_next_cuda",
    "rswa_debug_set_wait_limit_ns", "rswa_cache_kv_offsets",
    "rswa_qk_norm_rope", "rswa_qk_norm_rope_cached", "rswa_append_kv_rope",
    "rswa_decode_tree_workspace", "rswa_decode_tree", "rswa_commit_tree",
    "rswa_pages_footprint", "rswa_pages_create", "rswa_pages_destroy",
    "rswa_pages_append", "rswa_pages_attend_workspace", "rswa_pages_attend",
    "rswa_pages_weigh", "rswa_pages_evict_workspace", "rswa_pages_evict",
    "rswa_pages_kv_offsets", "rswa_pages_sync_status",
    "RswaRope", "RswaCache", "RswaBatch", "RswaPages",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
RSWA_F32, RSWA_BF16 = 0, 1
RSWA_EDEVICE = 6               # of rswa_status
_LIB = None

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_vp = ctypes.c_void_p
_c_size = ctypes.c_size_t



class _RopeStruct(ctypes.Structure):
    """struct rswa_rope of include/rswa.h."""
    _fields_ = [("q_weight", _c_vp), ("k_weight", _c_vp), ("inv_freq", _c_vp),
                ("eps", ctypes.c_float), ("rotary_dim", _c_int),
                ("interleaved", _c_int)]


_c_rope = ctypes.POINTER(_RopeStruct)


class _BatchStruct(ctypes.Structure):
    """struct rswa_batch of include/rswa.h."""
    _fields_ = [("table", _c_vp), ("lens", _c_vp), ("prefix", _c_vp), ("starts", _c_vp),
                ("max_pages", _c_i64), ("window", _c_i64), ("batch", _c_int)]


_c_batch = ctypes.POINTER(_BatchStruct)

_SIGNATURES = {
    "rswa_strerror": (ctypes.c_char_p, [_c_int]),
    "rswa_cache_footprint": (_c_int, [_c_i64, _c_i64, _c_int, _c_int, _c_int,
                                      _c_int, ctypes.POINTER(_c_size)]),
    "rswa_cache_create": (_c_int, [_c_i64, _c_i64, _c_int, _c_int, _c_int,
                                   _c_int, _c_vp, _c_size,
                                   ctypes.POINTER(_c_vp)]),
    "rswa_cache_footprint_gqa": (_c_int, [_c_i64, _c_i64, _c_int, _c_int, _c_int,
                                          _c_int, _c_int, ctypes.POINTER(_c_size)]),
    "rswa_cache_create_gqa": (_c_int, [_c_i64, _c_i64, _c_int, _c_int, _c_int,
                                       _c_int, _c_int, _c_vp, _c_size,
                                       ctypes.POINTER(_c_vp)]),
    "rswa_prefill_varlen": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                     ctypes.POINTER(_c_i64), ctypes.POINTER(_c_i64),
                                     _c_vp]),
    "rswa_cache_destroy": (_c_int, [_c_vp]),
    "rswa_prefill": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                              ctypes.POINTER(_c_i64), _c_i64, _c_vp]),
    "rswa_append_kv": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp]),
    "rswa_decode_step": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "rswa_decode_step_fused": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                        _c_vp, _c_vp]),
    "rswa_decode_step_fused_static": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp,
                                               _c_vp, _c_vp, _c_vp]),
    "rswa_decode_block": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp,
                                   _c_vp, _c_vp]),
    "rswa_cache_bytes": (_c_int, [_c_vp, _c_int, ctypes.POINTER(_c_size)]),
    "rswa_cache_len": (_c_int, [_c_vp, _c_int, ctypes.POINTER(_c_i64)]),
    "rswa_cache_get_t": (_c_int, [_c_vp, _c_int, ctypes.POINTER(_c_i64)]),
    "rswa_cache_set_t": (_c_int, [_c_vp, ctypes.POINTER(_c_i64), _c_vp]),
    "rswa_qk_norm_rope": (_c_int, [_c_rope, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp,
                                   _c_i64, _c_int, _c_int, _c_int, _c_int, _c_vp,
                                   _c_vp, _c_vp]),
    "rswa_qk_norm_rope_cached": (_c_int, [_c_vp, _c_rope, _c_vp, _c_i64, _c_vp,
                                          _c_i64, _c_vp, _c_i64, _c_vp, _c_vp,
                                          _c_vp]),
    "rswa_append_kv_rope": (_c_int, [_c_vp, _c_rope, _c_vp, _c_i64, _c_vp, _c_i64,
                                     _c_vp, _c_i64, _c_vp, _c_vp]),
    "rswa_decode_tree_workspace": (_c_int, [_c_vp, _c_i64,
                                            ctypes.POINTER(_c_size)]),
    "rswa_decode_tree": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64,
                                  _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "rswa_commit_tree": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64,
                                  _c_vp]),
    "rswa_pages_footprint": (_c_int, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int,
                                      ctypes.POINTER(_c_size)]),
    "rswa_pages_create": (_c_int, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int, _c_vp,
                                   _c_size, ctypes.POINTER(_c_vp)]),
    "rswa_pages_destroy": (_c_int, [_c_vp]),
    "rswa_pages_append": (_c_int, [_c_vp, _c_batch, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64,
                                   _c_vp]),
    "rswa_pages_attend_workspace": (_c_int, [_c_vp, _c_i64, ctypes.POINTER(_c_size)]),
    "rswa_pages_attend": (_c_int, [_c_vp, _c_batch, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp,
                                   _c_vp, _c_size, _c_vp]),
    "rswa_pages_weigh": (_c_int, [_c_vp, _c_batch, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp,
                                  ctypes.c_float, _c_vp]),
    "rswa_pages_evict_workspace": (_c_int, [_c_vp, _c_int, _c_i64, ctypes.POINTER(_c_size)]),
    "rswa_pages_evict": (_c_int, [_c_vp, _c_batch, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp,
                                  _c_vp, _c_vp, _c_size, _c_vp]),
    "rswa_pages_kv_offsets": (_c_int, [_c_vp, ctypes.POINTER(_c_size),
                                       ctypes.POINTER(_c_size)]),
    "rswa_pages_sync_status": (_c_int, [_c_vp]),
    "rswa_sync_status": (_c_int, [_c_vp]),
    "rswa_cache_kv_offsets": (_c_int, [_c_vp, ctypes.POINTER(_c_size),
                                       ctypes.POINTER(_c_size)]),
    "rswa_debug_fail_next_cuda": (None, [_c_int]),
    "rswa_debug_set_wait_limit_ns": (None, [ctypes.c_uint64]),
}


class RswaError(RuntimeError):
    """A non-zero rswa_status returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = load().rswa_strerror(status).decode()
        super().__init__(f"{where}: status {status} ({msg})")


def library_path() -> str:
    return os.path.join(_HERE, "librswa.so")


def declared_symbols() -> list:
    """Names declared RSWA_API in include/rswa.h."""
    import re
    with open(os.path.join(_ROOT, "include", "rswa.h")) as f:
        text = f.read()
    return re.findall(r"RSWA_API\s+[\w\s\*]+?\b(rswa_\w+)\s*\(", text)


def load():
    """Load librswa.so (built by ``__graft_entry__.build()``)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(status: int, where: str) -> None:
    if status != 0:
        raise RswaError(status, where)


def _ptr(t):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _row_ptr(t):
    """Device pointer of a CUDA tensor of rows with a stride."""
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _device_index(t) -> int:
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.get_device()


def _stream_of(stream, index: int):
    """The given stream, or the current one of device `index`."""
    if stream is None:
        return _current_stream(index)
    return getattr(stream, "cuda_stream", stream)


def _current_stream(index: int):
    """torch.cuda.current_stream(index).cuda_stream, without the Stream object
    (1.1 us of a call) where torch gives the pointer itself."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(index)


def _torch_stream(handle: int, index: int):
    """The torch stream of a handle (0 and cudaStreamLegacy: the default one)."""
    import torch
    if handle in (0, 1):
        return torch.cuda.default_stream(index)
    return torch.cuda.ExternalStream(handle, device=index)


def _current_device():
    """torch.cuda.current_device(), without its test for an initialised CUDA
    (0.2 us of a call): the caller has a CUDA tensor."""
    global _get_device
    if _get_device is None:
        import torch
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _get_device()


_raw_stream = _get_device = None


def _rows(t, shape, dtype, index, name):
    """(pointer, elements between rows) of rows of [heads][d] elements: a
    tensor [rows][heads][d] whose rows may be part of longer ones."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == index:
        stride, inner, last = t.stride()
        if last == 1 and (inner == shape[2] or shape[1] == 1):
            return t.data_ptr(), stride
    raise ValueError(f"{name}: expected {tuple(shape)} of {dtype} on CUDA device {index} with "
                     f"the heads of a row contiguous, got {tuple(t.shape)} of {t.dtype} on "
                     f"{t.device}, strides {t.stride()}")


def _dense(t, shape, dtype, index, name):
    """Pointer of a contiguous CUDA tensor of this shape and type."""
    if (t.shape == shape and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, contiguous on CUDA device "
                     f"{index}, got {tuple(t.shape)} of {t.dtype} on {t.device}, strides "
                     f"{t.stride()}")


def rswa_strerror(status: int) -> str:
    return load().rswa_strerror(status).decode()


def rswa_debug_fail_next_cuda(count: int) -> None:
    load().rswa_debug_fail_next_cuda(count)


def rswa_debug_set_wait_limit_ns(ns: int) -> None:
    load().rswa_debug_set_wait_limit_ns(int(ns))


def rswa_cache_footprint(m, n, heads, head_dim, batch, dtype) -> int:
    out = _c_size(0)
    _check(load().rswa_cache_footprint(m, n, heads, head_dim, batch, dtype,
                                       ctypes.byref(out)),
           "rswa_cache_footprint")
    return out.value


def rswa_cache_create(m, n, heads, head_dim, batch, dtype, buf):
    """Create a cache over the uint8 CUDA tensor ``buf``; returns the handle."""
    h = _c_vp()
    _check(load().rswa_cache_create(m, n, heads, head_dim, batch, dtype,
                                    _ptr(buf), buf.numel() * buf.element_size(),
                                    ctypes.byref(h)),
           "rswa_cache_create")
    return h.value


def rswa_cache_footprint_gqa(m, n, heads, kv_heads, head_dim, batch,
                             dtype) -> int:
    out = _c_size(0)
    _check(load().rswa_cache_footprint_gqa(m, n, heads, kv_heads, head_dim,
                                           batch, dtype, ctypes.byref(out)),
           "rswa_cache_footprint_gqa")
    return out.value


def rswa_cache_create_gqa(m, n, heads, kv_heads, head_dim, batch, dtype, buf):
    h = _c_vp()
    _check(load().rswa_cache_create_gqa(m, n, heads, kv_heads, head_dim, batch,
                                        dtype, _ptr(buf),
                                        buf.numel() * buf.element_size(),
                                        ctypes.byref(h)),
           "rswa_cache_create_gqa")
    return h.value


def rswa_cache_destroy(handle) -> None:
    _check(load().rswa_cache_destroy(handle), "rswa_cache_destroy")


def rswa_prefill(handle, Q, K, V, O, m_per_seq, T, stream=None) -> None:
    arr = (_c_i64 * len(m_per_seq))(*[int(x) for x in m_per_seq])
    _check(load().rswa_prefill(handle, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), arr,
                               int(T), _stream(stream)),
           "rswa_prefill")


def rswa_prefill_varlen(handle, Q, K, V, O, m_per_seq, t_per_seq,
                        stream=None) -> None:
    marr = (_c_i64 * len(m_per_seq))(*[int(x) for x in m_per_seq])
    tarr = (_c_i64 * len(t_per_seq))(*[int(x) for x in t_per_seq])
    _check(load().rswa_prefill_varlen(handle, _ptr(Q), _ptr(K), _ptr(V),
                                      _ptr(O), marr, tarr, _stream(stream)),
           "rswa_prefill_varlen")


def rswa_append_kv(handle, k, v, stream=None) -> None:
    _check(load().rswa_append_kv(handle, _ptr(k), _ptr(v), _stream(stream)),
           "rswa_append_kv")


def rswa_decode_step(handle, q, o, lse=None, stream=None) -> None:
    _check(load().rswa_decode_step(handle, _ptr(q), _ptr(o), _ptr(lse),
                                   _stream(stream)),
           "rswa_decode_step")


def rswa_decode_step_fused(handle, q, k, v, o, lse=None, stream=None) -> None:
    _check(load().rswa_decode_step_fused(handle, _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(o), _ptr(lse), _stream(stream)),
           "rswa_decode_step_fused")


def rswa_decode_step_fused_static(handle, q, k, v, o, lse=None,
                                  stream=None) -> None:
    """rswa_decode_step_fused with its split-K scratch in the library's fixed
    4 MiB device array instead of the cache buffer: the call allocates
    nothing (for callers that must not allocate device memory once decoding
    runs).  Overlapping calls race on that array."""
    _check(load().rswa_decode_step_fused_static(handle, _ptr(q), _ptr(k),
                                                _ptr(v), _ptr(o), _ptr(lse),
                                                _stream(stream)),
           "rswa_decode_step_fused_static")


def rswa_decode_block(handle, q, k, v, o, lse=None, stream=None) -> None:
    """q, k, v, o: [B][block][H][d]; lse: [B][block][H] or None."""
    _check(load().rswa_decode_block(handle, _ptr(q), _ptr(k), _ptr(v),
                                    int(q.shape[1]), _ptr(o), _ptr(lse),
                                    _stream(stream)),
           "rswa_decode_block")


def rswa_qk_norm_rope(rope, q, k, positions, q_out, k_out, stream=None) -> None:
    """rope: RswaRope; q, k: [rows][heads][d], the rows possibly part of longer
    ones (a fused projection's output); positions: int64 [rows]; q_out, k_out:
    contiguous, or q and k themselves."""
    shape, k_shape = q.shape, k.shape
    if len(shape) != 3 or len(k_shape) != 3:
        raise ValueError("q, k: expected [rows][heads][d]")
    index, dt, torch = q.get_device(), q.dtype, rope.torch
    rows, heads, d = shape
    kv_heads = k_shape[1]
    k_shape = (rows, kv_heads, d)
    if index < 0:
        raise ValueError("q: expected a CUDA tensor")
    code = RSWA_BF16 if dt is torch.bfloat16 else RSWA_F32 if dt is torch.float32 else -1
    if code < 0:
        raise ValueError(f"q, k: expected bfloat16 or float32, got {dt}")
    rope.check(d, dt, index)
    qp, qs = _rows(q, shape, dt, index, "q")
    kp, ks = _rows(k, k_shape, dt, index, "k")
    args = (rope.ref, qp, qs, kp, ks,
            _dense(positions, (rows,), torch.int64, index, "positions"), rows, heads, kv_heads,
            d, code, _dense(q_out, shape, dt, index, "q_out"),
            _dense(k_out, k_shape, dt, index, "k_out"), _stream_of(stream, index))
    if index == _current_device():
        status = load().rswa_qk_norm_rope(*args)
    else:
        with torch.cuda.device(index):
            status = load().rswa_qk_norm_rope(*args)
    if status:
        raise RswaError(status, "rswa_qk_norm_rope")


def rswa_qk_norm_rope_cached(handle, rope, q, q_stride, k, k_stride, offsets, tokens,
                             q_out, k_out, stream=None) -> None:
    """Pointers as tensors, strides in elements; RswaCache.qk_norm_rope checks
    shapes and types."""
    _check(load().rswa_qk_norm_rope_cached(
        handle, rope.ref, _row_ptr(q), q_stride, _row_ptr(k), k_stride,
        _ptr(offsets), tokens, _ptr(q_out), _ptr(k_out),
        _stream_of(stream, _device_index(q))), "rswa_qk_norm_rope_cached")


def rswa_append_kv_rope(handle, rope, q, q_stride, k, k_stride, v, v_stride, q_out,
                        stream=None) -> None:
    """Pointers as tensors, strides in elements; RswaCache.append_kv_rope
    checks shapes and types."""
    _check(load().rswa_append_kv_rope(
        handle, rope.ref, _row_ptr(q), q_stride, _row_ptr(k), k_stride,
        _row_ptr(v), v_stride, _ptr(q_out), _stream_of(stream, _device_index(q))),
        "rswa_append_kv_rope")


def rswa_decode_tree_workspace(handle, nodes: int) -> int:
    out = _c_size(0)
    _check(load().rswa_decode_tree_workspace(handle, nodes, ctypes.byref(out)),
           "rswa_decode_tree_workspace")
    return out.value


def rswa_decode_tree(handle, q, k, v, parents, o, lse, workspace, counts=None,
                     stream=None) -> None:
    """q, o: [B][nodes][H][d]; k, v: [B][nodes][H_kv][d]; parents: int32
    [B][nodes]; counts: int32 [B] or None; workspace: uint8 tensor."""
    _check(load().rswa_decode_tree(
        handle, _ptr(q), _ptr(k), _ptr(v), _ptr(parents), _ptr(counts),
        int(q.shape[1]), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
        _stream_of(stream, _device_index(q))), "rswa_decode_tree")


def rswa_commit_tree(handle, k, v, path, accepted, stream=None) -> None:
    """k, v: [B][nodes][H_kv][d]; path: int32 [B][max_path]; accepted: int32 [B]."""
    _check(load().rswa_commit_tree(
        handle, _ptr(k), _ptr(v), int(k.shape[1]), _ptr(path), _ptr(accepted),
        int(path.shape[1]), _stream_of(stream, _device_index(k))), "rswa_commit_tree")


def rswa_pages_footprint(pages, page_size, heads, kv_heads, head_dim, dtype) -> int:
    out = _c_size(0)
    _check(load().rswa_pages_footprint(pages, page_size, heads, kv_heads, head_dim, dtype,
                                       ctypes.byref(out)), "rswa_pages_footprint")
    return out.value


def rswa_pages_create(pages, page_size, heads, kv_heads, head_dim, dtype, buf):
    """Create a pool over the uint8 CUDA tensor ``buf``; returns the handle."""
    h = _c_vp()
    _check(load().rswa_pages_create(pages, page_size, heads, kv_heads, head_dim, dtype,
                                    _ptr(buf), buf.numel() * buf.element_size(),
                                    ctypes.byref(h)), "rswa_pages_create")
    return h.value


def rswa_pages_destroy(handle) -> None:
    _check(load().rswa_pages_destroy(handle), "rswa_pages_destroy")


def rswa_pages_append(handle, batch, k, k_stride, v, v_stride, stream=None) -> None:
    """batch: RswaBatch; pointers as tensors, strides in elements;
    RswaPages.append checks shapes and types."""
    _check(load().rswa_pages_append(
        handle, batch.ref, int(k.shape[0]), _row_ptr(k), k_stride, _row_ptr(v), v_stride,
        _stream_of(stream, _device_index(k))), "rswa_pages_append")


def rswa_pages_attend_workspace(handle, rows: int) -> int:
    out = _c_size(0)
    _check(load().rswa_pages_attend_workspace(handle, rows, ctypes.byref(out)),
           "rswa_pages_attend_workspace")
    return out.value


def rswa_pages_attend(handle, batch, q, q_stride, o, workspace, lse=None, stream=None) -> None:
    """RswaPages.attend checks shapes and types; workspace: zeroed uint8 tensor."""
    _check(load().rswa_pages_attend(
        handle, batch.ref, int(q.shape[0]), _row_ptr(q), q_stride, _ptr(o), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream_of(stream, _device_index(q))),
        "rswa_pages_attend")


def rswa_pages_weigh(handle, batch, q, q_stride, lse, weights, decay=1.0, stream=None) -> None:
    """RswaPages.weigh checks shapes and types."""
    _check(load().rswa_pages_weigh(
        handle, batch.ref, int(q.shape[0]), _row_ptr(q), q_stride, _ptr(lse), _ptr(weights),
        decay, _stream_of(stream, _device_index(weights))), "rswa_pages_weigh")


def rswa_pages_evict_workspace(handle, batch: int, budget: int) -> int:
    out = _c_size(0)
    _check(load().rswa_pages_evict_workspace(handle, batch, budget, ctypes.byref(out)),
           "rswa_pages_evict_workspace")
    return out.value


def rswa_pages_evict(handle, batch, weights, budget, first, last, weights_out, workspace,
                     table_out=None, kept=None, stream=None) -> None:
    """RswaPages.evict checks shapes and types."""
    _check(load().rswa_pages_evict(
        handle, batch.ref, _ptr(weights), budget, first, last, _ptr(table_out),
        _ptr(weights_out), _ptr(kept), _ptr(workspace), workspace.numel(),
        _stream_of(stream, _device_index(weights))), "rswa_pages_evict")


def rswa_pages_kv_offsets(handle):
    ko, vo = _c_size(0), _c_size(0)
    _check(load().rswa_pages_kv_offsets(handle, ctypes.byref(ko), ctypes.byref(vo)),
           "rswa_pages_kv_offsets")
    return ko.value, vo.value


def rswa_pages_sync_status(handle) -> int:
    """Returns the status code (does not raise)."""
    return load().rswa_pages_sync_status(handle)


def rswa_cache_bytes(handle, b: int) -> int:
    out = _c_size(0)
    _check(load().rswa_cache_bytes(handle, b, ctypes.byref(out)),
           "rswa_cache_bytes")
    return out.value


def rswa_cache_len(handle, b: int) -> int:
    out = _c_i64(0)
    _check(load().rswa_cache_len(handle, b, ctypes.byref(out)), "rswa_cache_len")
    return out.value


def rswa_cache_get_t(handle, b: int) -> int:
    out = _c_i64(0)
    _check(load().rswa_cache_get_t(handle, b, ctypes.byref(out)),
           "rswa_cache_get_t")
    return out.value


def rswa_cache_set_t(handle, t_per_seq, stream=None) -> None:
    arr = (_c_i64 * len(t_per_seq))(*[int(x) for x in t_per_seq])
    _check(load().rswa_cache_set_t(handle, arr, _stream(stream)),
           "rswa_cache_set_t")


def rswa_cache_kv_offsets(handle):
    ko, vo = _c_size(0), _c_size(0)
    _check(load().rswa_cache_kv_offsets(handle, ctypes.byref(ko),
                                        ctypes.byref(vo)),
           "rswa_cache_kv_offsets")
    return ko.value, vo.value


def rswa_sync_status(handle) -> int:
    """Returns the status code (does not raise)."""
    return load().rswa_sync_status(handle)


class RswaRope:
    """The norm and rotation of a layer's query and key heads (struct
    rswa_rope), with the tensors it points to.

    inv_freq: float64 CUDA tensor of radians per position, one for each rotated
    pair (2 * len elements of a head are rotated), or None for no rotation;
    q_weight, k_weight: [head_dim] norm weights in the heads' type, or None for
    no norm.
    """

    def __init__(self, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False):
        import torch
        self.torch = torch
        self.inv_freq, self.q_weight, self.k_weight = inv_freq, q_weight, k_weight
        if inv_freq is not None and (inv_freq.dtype != torch.float64
                                     or inv_freq.dim() != 1):
            raise ValueError("inv_freq: expected a float64 vector")
        weights = [w for w in (q_weight, k_weight) if w is not None]
        if any(w.dim() != 1 for w in weights):
            raise ValueError("q_weight, k_weight: expected vectors")
        tensors = weights + ([] if inv_freq is None else [inv_freq])
        if len({_device_index(t) for t in tensors}) > 1:
            raise ValueError("inv_freq and weights: different devices")
        self.rotary_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
        self._struct = _RopeStruct(_ptr(q_weight), _ptr(k_weight),
                                   _ptr(inv_freq) if self.rotary_dim else None,
                                   float(eps), self.rotary_dim, int(bool(interleaved)))
        self.ref = ctypes.byref(self._struct)
        # what its calls' heads have to be
        self._need = [(w.numel(), w.dtype) for w in weights]
        self._index = _device_index(tensors[0]) if tensors else None
        self._fits = None               # the last heads that passed

    def check(self, d, dtype, index):
        """Raise unless it fits heads of d elements of dtype on device index."""
        if (d, dtype, index) == self._fits:
            return
        for need in self._need:
            if need != (d, dtype):
                raise ValueError(f"rope: weights of {need[0]} {need[1]}, heads of "
                                 f"{d} {dtype}")
        if self._index is not None and self._index != index:
            raise ValueError("rope: on another device than the heads")
        self._fits = (d, dtype, index)


class RswaCache:
    """A cache plus the torch-allocated device buffer that backs it."""

    def __init__(self, m, n, heads, head_dim, batch, dtype, device="cuda",
                 kv_heads=None):
        import torch
        self.m, self.n, self.heads, self.head_dim = m, n, heads, head_dim
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.batch, self.dtype = batch, dtype
        nbytes = rswa_cache_footprint_gqa(m, n, heads, self.kv_heads, head_dim,
                                          batch, dtype)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        # its block may be one that the current stream still writes, and the state is
        # zeroed on another stream
        torch.cuda.current_stream(self.buf.device).synchronize()
        self.handle = rswa_cache_create_gqa(m, n, heads, self.kv_heads,
                                            head_dim, batch, dtype, self.buf)
        # what the checks of the draft-and-verify calls compare with
        self._shape = (batch, heads, self.kv_heads, head_dim,
                       torch.float32 if dtype == RSWA_F32 else torch.bfloat16,
                       self.buf.get_device())
        self._int32, self._float32 = torch.int32, torch.float32
        # decode_tree's own workspaces, by node count and stream; all stay, as
        # captured graphs hold them
        self._tree_ws = {}
        self._tree_at = {}              # and their pointers and sizes

    def close(self):
        if self.handle is not None:
            rswa_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # thin forwards
    def prefill(self, Q, K, V, O, m_per_seq, T, stream=None):
        rswa_prefill(self.handle, Q, K, V, O, m_per_seq, T, stream)

    def prefill_varlen(self, Q, K, V, O, m_per_seq, t_per_seq, stream=None):
        rswa_prefill_varlen(self.handle, Q, K, V, O, m_per_seq, t_per_seq,
                            stream)

    def append_kv(self, k, v, stream=None):
        rswa_append_kv(self.handle, k, v, stream)

    def decode_step(self, q, o, lse=None, stream=None):
        rswa_decode_step(self.handle, q, o, lse, stream)

    def decode_step_fused(self, q, k, v, o, lse=None, stream=None):
        rswa_decode_step_fused(self.handle, q, k, v, o, lse, stream)

    def decode_block(self, q, k, v, o, lse=None, stream=None):
        rswa_decode_block(self.handle, q, k, v, o, lse, stream)

    def qk_norm_rope(self, rope, q, k, q_out, k_out, offsets=None, stream=None):
        """Norm and rotate the heads of the next tokens of every sequence: q, k
        of [B * tokens][heads][d] rows (possibly part of longer ones), at
        positions m_b + t_b + offsets (int32 [B][tokens]; None: 0, 1, ...)."""
        B, H, Hkv, d, dt, ix = self._shape
        rows = q.shape[0]
        if rows % B:
            raise ValueError("q: expected batch * tokens rows")
        rope.check(d, dt, ix)
        qp, qs = _rows(q, (rows, H, d), dt, ix, "q")
        kp, ks = _rows(k, (rows, Hkv, d), dt, ix, "k")
        op = None if offsets is None else _dense(offsets, (B, rows // B), self._int32, ix,
                                                 "offsets")
        status = load().rswa_qk_norm_rope_cached(
            self.handle, rope.ref, qp, qs, kp, ks, op, rows // B,
            _dense(q_out, (rows, H, d), dt, ix, "q_out"),
            _dense(k_out, (rows, Hkv, d), dt, ix, "k_out"), _stream_of(stream, ix))
        if status:
            raise RswaError(status, "rswa_qk_norm_rope_cached")

    def append_kv_rope(self, rope, q, k, v, q_out, stream=None):
        """append_kv with the norm and rotation on the way: q, k, v of
        [B][heads][d] rows (possibly part of longer ones); q_out takes the
        normed and rotated queries for decode_step."""
        B, H, Hkv, d, dt, ix = self._shape
        rope.check(d, dt, ix)
        qp, qs = _rows(q, (B, H, d), dt, ix, "q")
        kp, ks = _rows(k, (B, Hkv, d), dt, ix, "k")
        vp, vs = _rows(v, (B, Hkv, d), dt, ix, "v")
        status = load().rswa_append_kv_rope(
            self.handle, rope.ref, qp, qs, kp, ks, vp, vs,
            _dense(q_out, (B, H, d), dt, ix, "q_out"), _stream_of(stream, ix))
        if status:
            raise RswaError(status, "rswa_append_kv_rope")

    def tree_workspace(self, nodes):
        """A workspace for decode_tree calls of up to `nodes` nodes, like any
        tensor made on torch's current stream."""
        import torch
        return torch.empty(rswa_decode_tree_workspace(self.handle, nodes),
                           dtype=torch.uint8, device=self.buf.device)

    def decode_tree(self, q, k, v, parents, o, lse=None, counts=None, workspace=None,
                    stream=None):
        """Attention of a tree of drafted tokens per sequence over the cache
        (see rswa_decode_tree).  workspace: from tree_workspace; None: one the
        cache keeps for the stream; a capture takes one that a call before it
        has made."""
        B, H, Hkv, d, dt, ix = self._shape
        nodes = q.shape[1]
        i32 = self._int32
        qp = _dense(q, (B, nodes, H, d), dt, ix, "q")
        kp = _dense(k, (B, nodes, Hkv, d), dt, ix, "k")
        vp = _dense(v, (B, nodes, Hkv, d), dt, ix, "v")
        pp = _dense(parents, (B, nodes), i32, ix, "parents")
        op = _dense(o, (B, nodes, H, d), dt, ix, "o")
        lp = None if lse is None else _dense(lse, (B, nodes, H), self._float32, ix, "lse")
        cp = None if counts is None else _dense(counts, (B,), i32, ix, "counts")
        at = _stream_of(stream, ix)
        if workspace is None:
            wp, size = self._tree_at.get((nodes, at)) or self._own_workspace(nodes, at)
        elif workspace.get_device() != ix:
            raise ValueError(f"workspace: expected a tensor on CUDA device {ix}")
        else:
            wp, size = _ptr(workspace), workspace.numel()
        status = load().rswa_decode_tree(
            self.handle, qp, kp, vp, pp, cp, nodes, op, lp, wp, size, at)
        if status:
            raise RswaError(status, "rswa_decode_tree")

    def _own_workspace(self, nodes, stream):
        """(pointer, bytes) of the cache's workspace for trees of `nodes` nodes on a
        stream (handle): made by the first call there that needs one (or a larger one), from the
        stream's own pool, so that torch's allocator neither hands the cache a
        block that other queued work still uses nor, once the cache is gone,
        others one that the stream's queued calls do.  A capture takes one made
        before it: calls on one cache are ordered, so it need not be its own."""
        import torch
        stream = getattr(stream, "value", stream) or 0
        need = rswa_decode_tree_workspace(self.handle, nodes)
        capturing = torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(_torch_stream(stream, self.buf.get_device())):
            if capturing or torch.cuda.is_current_stream_capturing():
                have = next((w for w in self._tree_ws.values() if w.numel() >= need), None)
                if have is None:
                    raise ValueError("decode_tree: no workspace of the cache's own yet: call it "
                                     "once before the capture, or pass one")
                return have.data_ptr(), have.numel()
            have = next((w for (_, at), w in self._tree_ws.items()
                         if at == stream and w.numel() >= need), None)
            if have is None:
                have = self.tree_workspace(nodes)
        self._tree_ws[nodes, stream] = have
        self._tree_at[nodes, stream] = have.data_ptr(), have.numel()
        return self._tree_at[nodes, stream]

    def commit_tree(self, k, v, path, accepted, stream=None):
        """Append the accepted nodes path[b][:accepted[b]] of a tree."""
        B, _, Hkv, d, dt, ix = self._shape
        nodes, most = k.shape[1], path.shape[-1]
        status = load().rswa_commit_tree(
            self.handle, _dense(k, (B, nodes, Hkv, d), dt, ix, "k"),
            _dense(v, (B, nodes, Hkv, d), dt, ix, "v"), nodes,
            _dense(path, (B, most), self._int32, ix, "path"),
            _dense(accepted, (B,), self._int32, ix, "accepted"), most, _stream_of(stream, ix))
        if status:
            raise RswaError(status, "rswa_commit_tree")

    def cache_bytes(self, b):
        return rswa_cache_bytes(self.handle, b)

    def cache_len(self, b):
        return rswa_cache_len(self.handle, b)

    def get_t(self, b):
        return rswa_cache_get_t(self.handle, b)

    def set_t(self, t_per_seq, stream=None):
        rswa_cache_set_t(self.handle, t_per_seq, stream)

    def sync_status(self):
        return rswa_sync_status(self.handle)

    def slabs(self):
        """(K, V) views of the cache slabs [B][H_kv][m + n][d] (for tests)."""
        import torch
        tdt = torch.float32 if self.dtype == RSWA_F32 else torch.bfloat16
        elt = 4 if self.dtype == RSWA_F32 else 2
        B, H, R, d = self.batch, self.kv_heads, self.m + self.n, self.head_dim
        nb = B * H * R * d * elt
        ko, vo = rswa_cache_kv_offsets(self.handle)
        Kt = self.buf[ko:ko + nb].view(tdt).view(B, H, R, d)
        Vt = self.buf[vo:vo + nb].view(tdt).view(B, H, R, d)
        return Kt, Vt


class RswaBatch:
    """The sequences of the calls on a paged cache (struct rswa_batch), with the
    tensors it points to: int32 CUDA tensors that the calls read when they run, so
    that a step may rewrite them in place.

    table: [B][max_pages], the page of each page_size tokens; lens: [B] tokens,
    the chunk's included; starts: [B + 1], the rows of the chunk that each sequence
    has, or None for the same number each; prefix: [B] first tokens that stay
    visible, or None; window: tokens that a token sees back, itself included, or
    None for all.
    """

    def __init__(self, table, lens, starts=None, prefix=None, window=None):
        import torch
        if table.dim() != 2:
            raise ValueError("table: expected [batch][max_pages]")
        B = table.shape[0]
        index = _device_index(table)
        self.table, self.lens, self.starts, self.prefix = table, lens, starts, prefix
        self.shape, self.index = (B, table.shape[1]), index

        def ints(t, shape, name):
            return None if t is None else _dense(t, shape, torch.int32, index, name)

        if window is not None and window < 1:
            raise ValueError("window: expected at least 1")
        self._struct = _BatchStruct(
            ints(table, self.shape, "table"), ints(lens, (B,), "lens"),
            ints(prefix, (B,), "prefix"), ints(starts, (B + 1,), "starts"), table.shape[1],
            1 << 30 if window is None else min(int(window), 1 << 30), B)
        self.ref = ctypes.byref(self._struct)


class _Workspaces:
    """A handle's own workspaces: one for each stream that a call runs on, made (or
    made larger) by the first call there that needs it, from the stream's own pool,
    so that torch's allocator neither hands out a block that other queued work still
    uses nor, once the handle is gone, gives others one that the stream's queued
    calls do.  All stay, as captured graphs hold them."""

    def __init__(self, index, what):
        self.index, self.what = index, what
        self.all = []                   # (stream, tensor)
        self.at = {}                    # stream: (pointer, bytes) of its largest

    def get(self, stream, need):
        """(pointer, bytes) of one of at least `need` bytes for a stream (handle)."""
        stream = getattr(stream, "value", stream) or 0
        have = self.at.get(stream)
        if have is not None and have[1] >= need:
            return have
        import torch
        capturing = torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(_torch_stream(stream, self.index)):
            if capturing or torch.cuda.is_current_stream_capturing():
                raise ValueError(f"{self.what}: no workspace of its own for this stream yet: "
                                 f"call it there once before the capture, or pass one")
            w = torch.zeros(need, dtype=torch.uint8, device=torch.device("cuda", self.index))
        self.all.append((stream, w))
        self.at[stream] = (w.data_ptr(), w.numel())
        return self.at[stream]

    def zero(self):
        """All of them as they were made; waits for it."""
        import torch
        for _, w in self.all:
            w.zero_()
        torch.cuda.synchronize(self.index)


_NO_WORKSPACE = (None, 0, -1)


class RswaPages:
    """A paged cache: a pool of pages plus the torch-allocated buffer behind it."""

    def __init__(self, pages, page_size, heads, head_dim, dtype, device="cuda", kv_heads=None):
        import torch
        self.pages, self.page_size, self.heads, self.head_dim = pages, page_size, heads, head_dim
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.dtype, self.handle = dtype, None
        nbytes = rswa_pages_footprint(pages, page_size, heads, self.kv_heads, head_dim, dtype)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ix = self.buf.get_device()
        with torch.cuda.device(ix):
            # its block may be one that the current stream still writes, and the flag is
            # zeroed on another stream
            torch.cuda.current_stream().synchronize()
            self.handle = rswa_pages_create(pages, page_size, heads, self.kv_heads, head_dim,
                                            dtype, self.buf)
        self._shape = (heads, self.kv_heads, head_dim,
                       torch.float32 if dtype == RSWA_F32 else torch.bfloat16, ix)
        self._int32, self._float32 = torch.int32, torch.float32
        self._attend_ws = _Workspaces(ix, "attend")
        self._evict_ws = _Workspaces(ix, "evict")
        self._attend_at = {}            # stream: (pointer, bytes, most rows) of attend's
        self._evict_need = {}
        self._lib = load()

    def close(self):
        if self.handle is not None:
            rswa_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_batch(self, batch):
        if batch.index != self._shape[4]:
            raise ValueError("batch: on another device than the pages")

    def append(self, batch, k, v, stream=None):
        """Store the chunk's keys and values: k, v of [rows][kv_heads][d] rows
        (possibly part of longer ones)."""
        H, Hkv, d, dt, ix = self._shape
        rows = k.shape[0]
        self._check_batch(batch)
        kp, ks = _rows(k, (rows, Hkv, d), dt, ix, "k")
        vp, vs = _rows(v, (rows, Hkv, d), dt, ix, "v")
        status = self._lib.rswa_pages_append(self.handle, batch.ref, rows, kp, ks, vp, vs,
                                             _stream_of(stream, ix))
        if status:
            raise RswaError(status, "rswa_pages_append")

    def attend_workspace(self, rows):
        """A workspace for attend calls of up to `rows` rows, like any tensor made on
        torch's current stream.  The calls of several pools (a model's layers) that run
        one after the other can share one: the largest of theirs serves all, where each
        pool keeps up to 40 MB for a stream by itself."""
        import torch
        return torch.zeros(rswa_pages_attend_workspace(self.handle, rows),
                           dtype=torch.uint8, device=self.buf.device)

    def attend(self, batch, q, o, lse=None, workspace=None, stream=None):
        """Attention of the chunk's rows over the pages (see rswa_pages_attend): q
        of [rows][heads][d] rows (possibly part of longer ones), o contiguous, lse
        float32 [rows][heads] or None.  workspace: from attend_workspace; None: one
        kept for the stream; a capture takes one that a call there has made.  So
        graphs captured on one stream, and the calls made on it, share theirs: where
        they may run at the same time, pass each a workspace of its own."""
        H, Hkv, d, dt, ix = self._shape
        rows = q.shape[0]
        self._check_batch(batch)
        qp, qs = _rows(q, (rows, H, d), dt, ix, "q")
        op = _dense(o, (rows, H, d), dt, ix, "o")
        lp = None if lse is None else _dense(lse, (rows, H), self._float32, ix, "lse")
        at = _stream_of(stream, ix)
        if workspace is None:
            # what is enough for these rows, if a call on this stream has had as many
            wp, size, most = self._attend_at.get(at, _NO_WORKSPACE)
            if rows > most:
                wp, size = self._attend_ws.get(at, rswa_pages_attend_workspace(self.handle, rows))
                self._attend_at[at] = wp, size, rows
        elif workspace.get_device() != ix:
            raise ValueError(f"workspace: expected a tensor on CUDA device {ix}")
        else:
            wp, size = _ptr(workspace), workspace.numel()
        status = self._lib.rswa_pages_attend(self.handle, batch.ref, rows, qp, qs, op, lp, wp,
                                             size, at)
        if status:
            raise RswaError(status, "rswa_pages_attend")

    def _weights(self, t, batch, name):
        B, width = batch.shape
        return _dense(t, (B, self.kv_heads, width * self.page_size), self._float32,
                      self._shape[4], name)

    def weigh(self, batch, q, lse, weights, decay=1.0, stream=None):
        """Add the attention weights that the cached tokens receive from the
        chunk's rows: weights float32 [B][kv_heads][max_pages * page_size] =
        decay * weights + what they receive; lse as attend gave it."""
        H, Hkv, d, dt, ix = self._shape
        rows = q.shape[0]
        self._check_batch(batch)
        qp, qs = _rows(q, (rows, H, d), dt, ix, "q")
        status = self._lib.rswa_pages_weigh(
            self.handle, batch.ref, rows, qp, qs, _dense(lse, (rows, H), self._float32, ix, "lse"),
            self._weights(weights, batch, "weights"), decay, _stream_of(stream, ix))
        if status:
            raise RswaError(status, "rswa_pages_weigh")

    def evict_workspace(self, sequences, budget):
        """A workspace for evict calls of so many sequences and this budget, like any
        tensor made on torch's current stream."""
        import torch
        return torch.empty(rswa_pages_evict_workspace(self.handle, sequences, budget),
                           dtype=torch.uint8, device=self.buf.device)

    def evict(self, batch, weights, budget, first=0, last=0, table_out=None, weights_out=None,
              kept=None, workspace=None, stream=None):
        """Cut every sequence down to `budget` tokens: its first and last ones and
        the heaviest of the others, in their order (see rswa_pages_evict).  In
        place, or to the pages of table_out; weights_out: weights itself where
        None; kept: int32 [B][kv_heads][budget] for the tokens' former indices;
        workspace: from evict_workspace, None: one kept for the stream, as attend's."""
        ix = self._shape[4]
        B, width = batch.shape
        self._check_batch(batch)
        wp = self._weights(weights, batch, "weights")
        wo = wp if weights_out is None else self._weights(weights_out, batch, "weights_out")
        tp = None if table_out is None else _dense(table_out, (B, width), self._int32, ix,
                                                   "table_out")
        kp = None if kept is None else _dense(kept, (B, self.kv_heads, budget), self._int32, ix,
                                              "kept")
        at = _stream_of(stream, ix)
        if workspace is None:
            need = self._evict_need.get((B, budget))
            if need is None:
                need = rswa_pages_evict_workspace(self.handle, B, budget)
                self._evict_need[B, budget] = need
            sp, size = self._evict_ws.get(at, need)
        elif workspace.get_device() != ix:
            raise ValueError(f"workspace: expected a tensor on CUDA device {ix}")
        else:
            sp, size = _ptr(workspace), workspace.numel()
        status = self._lib.rswa_pages_evict(self.handle, batch.ref, wp, budget, first, last, tp,
                                            wo, kp, sp, size, at)
        if status:
            raise RswaError(status, "rswa_pages_evict")

    def sync_status(self):
        """rswa_pages_sync_status: waits for the device; the status code, not raised.
        After RSWA_EDEVICE the pool's own workspaces are zeroed again; one that the
        caller passes is the caller's to zero."""
        status = rswa_pages_sync_status(self.handle)
        if status == RSWA_EDEVICE:
            self._attend_ws.zero()
        return status

    def slabs(self):
        """(K, V) views of the pools [pages][kv_heads][page_size][d]."""
        H, Hkv, d, tdt, ix = self._shape
        shape = (self.pages, Hkv, self.page_size, d)
        nb = self.pages * Hkv * self.page_size * d * (4 if self.dtype == RSWA_F32 else 2)
        ko, vo = rswa_pages_kv_offsets(self.handle)
        return (self.buf[ko:ko + nb].view(tdt).view(shape),
                self.buf[vo:vo + nb].view(tdt).view(shape))
