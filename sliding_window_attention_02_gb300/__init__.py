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
    "RswaRope", "RswaCache",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
RSWA_F32, RSWA_BF16 = 0, 1
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
