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
        import torch
        return torch.cuda.current_stream(index).cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _rows(t, heads, d, dtype, index, name):
    """(pointer, elements between rows) of rows of [heads][d] elements: a
    tensor [rows][heads][d] whose rows may be part of longer ones."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d or t.dtype != dtype:
        raise ValueError(f"{name}: expected [rows][{heads}][{d}] of {dtype}, "
                         f"got {tuple(t.shape)} of {t.dtype}")
    s = t.stride()
    if (s[2] != 1 and d > 1) or (s[1] != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a CUDA tensor of device {index}")
    return t.data_ptr(), s[0]


def _dense(t, shape, dtype, index, name):
    """Pointer of a contiguous CUDA tensor of this shape and type."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {tuple(shape)} of {dtype}, got "
                         f"{tuple(t.shape)} of {t.dtype}")
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of device {index}")
    return t.data_ptr()


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
    import torch
    index = _device_index(q)
    rows, heads, d = q.shape
    kv_heads = k.shape[1] if k.dim() == 3 else 0
    dt = q.dtype
    if k.shape[0] != rows:
        raise ValueError("q and k: different numbers of rows")
    rope.check(d, dt, index)
    qp, qs = _rows(q, heads, d, dt, index, "q")
    kp, ks = _rows(k, kv_heads, d, dt, index, "k")
    args = (rope.ref, qp, qs, kp, ks,
            _dense(positions, (rows,), torch.int64, index, "positions"), rows, heads,
            kv_heads, d, _rswa_dtype(dt),
            _dense(q_out, (rows, heads, d), dt, index, "q_out"),
            _dense(k_out, (rows, kv_heads, d), dt, index, "k_out"))
    if index == torch.cuda.current_device():
        _check(load().rswa_qk_norm_rope(*args, _stream_of(stream, index)),
               "rswa_qk_norm_rope")
    else:
        with torch.cuda.device(index):
            _check(load().rswa_qk_norm_rope(*args, _stream_of(stream, index)),
                   "rswa_qk_norm_rope")


def rswa_qk_norm_rope_cached(handle, rope, q, q_stride, k, k_stride, offsets, tokens,
                             q_out, k_out, stream=None) -> None:
    """Pointers as tensors, strides in elements; RswaCache.qk_norm_rope checks
    shapes and types."""
    _check(load().rswa_qk_norm_rope_cached(
        handle, rope.ref, q.data_ptr(), q_stride, k.data_ptr(), k_stride,
        _ptr(offsets), tokens, _ptr(q_out), _ptr(k_out),
        _stream_of(stream, _device_index(q))), "rswa_qk_norm_rope_cached")


def rswa_append_kv_rope(handle, rope, q, q_stride, k, k_stride, v, v_stride, q_out,
                        stream=None) -> None:
    """Pointers as tensors, strides in elements; RswaCache.append_kv_rope
    checks shapes and types."""
    _check(load().rswa_append_kv_rope(
        handle, rope.ref, q.data_ptr(), q_stride, k.data_ptr(), k_stride,
        v.data_ptr(), v_stride, _ptr(q_out), _stream_of(stream, _device_index(q))),
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


def _rswa_dtype(dt) -> int:
    import torch
    if dt == torch.bfloat16:
        return RSWA_BF16
    if dt == torch.float32:
        return RSWA_F32
    raise ValueError(f"expected bfloat16 or float32, got {dt}")


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

    def check(self, d, dtype, index):
        """Raise unless it fits heads of d elements of dtype on device index."""
        for need in self._need:
            if need != (d, dtype):
                raise ValueError(f"rope: weights of {need[0]} {need[1]}, heads of "
                                 f"{d} {dtype}")
        if self._index is not None and self._index != index:
            raise ValueError("rope: on another device than the heads")


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
        self._torch_dtype = torch.float32 if dtype == RSWA_F32 else torch.bfloat16
        self._index = self.buf.get_device()
        self._tree_ws = []          # smaller ones stay: captured graphs hold them

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
        import torch
        H, Hkv, d, dt, ix = (self.heads, self.kv_heads, self.head_dim,
                             self._torch_dtype, self._index)
        rope.check(d, dt, ix)
        _, qs = _rows(q, H, d, dt, ix, "q")
        _, ks = _rows(k, Hkv, d, dt, ix, "k")
        rows = q.shape[0]
        if rows % self.batch or k.shape[0] != rows:
            raise ValueError("q, k: expected batch * tokens rows each")
        _dense(q_out, (rows, H, d), dt, ix, "q_out")
        _dense(k_out, (rows, Hkv, d), dt, ix, "k_out")
        if offsets is not None:
            _dense(offsets, (self.batch, rows // self.batch), torch.int32, ix, "offsets")
        rswa_qk_norm_rope_cached(self.handle, rope, q, qs, k, ks, offsets,
                                 rows // self.batch, q_out, k_out, stream)

    def append_kv_rope(self, rope, q, k, v, q_out, stream=None):
        """append_kv with the norm and rotation on the way: q, k, v of
        [B][heads][d] rows (possibly part of longer ones); q_out takes the
        normed and rotated queries for decode_step."""
        H, Hkv, d, dt, ix = (self.heads, self.kv_heads, self.head_dim,
                             self._torch_dtype, self._index)
        rope.check(d, dt, ix)
        B = self.batch
        _, qs = _rows(q, H, d, dt, ix, "q")
        _, ks = _rows(k, Hkv, d, dt, ix, "k")
        _, vs = _rows(v, Hkv, d, dt, ix, "v")
        if q.shape[0] != B or k.shape[0] != B or v.shape[0] != B:
            raise ValueError(f"q, k, v: expected {B} rows each")
        _dense(q_out, (B, H, d), dt, ix, "q_out")
        rswa_append_kv_rope(self.handle, rope, q, qs, k, ks, v, vs, q_out, stream)

    def tree_workspace(self, nodes):
        """A workspace for decode_tree calls of up to `nodes` nodes."""
        import torch
        return torch.empty(rswa_decode_tree_workspace(self.handle, nodes),
                           dtype=torch.uint8, device=self.buf.device)

    def decode_tree(self, q, k, v, parents, o, lse=None, counts=None, workspace=None,
                    stream=None):
        """Attention of a tree of drafted tokens per sequence over the cache
        (see rswa_decode_tree).  workspace: from tree_workspace; None: one the
        cache keeps, which has to exist before a stream capture (by a call
        outside it) and serves calls that do not overlap."""
        import torch
        B, H, Hkv, d, dt, ix = (self.batch, self.heads, self.kv_heads, self.head_dim,
                                self._torch_dtype, self._index)
        nodes = q.shape[1]
        _dense(q, (B, nodes, H, d), dt, ix, "q")
        _dense(k, (B, nodes, Hkv, d), dt, ix, "k")
        _dense(v, (B, nodes, Hkv, d), dt, ix, "v")
        _dense(parents, (B, nodes), torch.int32, ix, "parents")
        _dense(o, (B, nodes, H, d), dt, ix, "o")
        if lse is not None:
            _dense(lse, (B, nodes, H), torch.float32, ix, "lse")
        if counts is not None:
            _dense(counts, (B,), torch.int32, ix, "counts")
        if workspace is None:
            need = rswa_decode_tree_workspace(self.handle, nodes)
            if not self._tree_ws or self._tree_ws[-1].numel() < need:
                if torch.cuda.is_current_stream_capturing():
                    raise ValueError("decode_tree: no workspace of the cache's own yet: "
                                     "call it once before the capture, or pass one")
                self._tree_ws.append(self.tree_workspace(nodes))
            workspace = self._tree_ws[-1]
        rswa_decode_tree(self.handle, q, k, v, parents, o, lse, workspace, counts, stream)

    def commit_tree(self, k, v, path, accepted, stream=None):
        """Append the accepted nodes path[b][:accepted[b]] of a tree."""
        import torch
        B, ix = self.batch, self._index
        shape = (B, k.shape[1], self.kv_heads, self.head_dim)
        _dense(k, shape, self._torch_dtype, ix, "k")
        _dense(v, shape, self._torch_dtype, ix, "v")
        _dense(path, (B, path.shape[1]), torch.int32, ix, "path")
        _dense(accepted, (B,), torch.int32, ix, "accepted")
        rswa_commit_tree(self.handle, k, v, path, accepted, stream)

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
