"""Python binding of libqwm.so, the B200 QuantWM 2-bit KV-cache library.

Argument marshalling only: every function forwards to the C entry point of the
same name declared in ``include/qwm.h``; every step of the computation runs in
the library's CUDA kernels.  PyTorch provides device memory and streams.  There
is no CPU fallback: a missing library or a tensor that is not on a CUDA device
raises.

Tensors Q, K, V, O are token-major ``[n][heads][head_dim]`` ``torch.bfloat16``
(contiguous, CUDA).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

__all__ = [
    "QwmError", "qwm_config", "qwm_sizes", "qwm_buffers", "qwm_cache", "BUFFER_NAMES",
    "lib", "qwm_abi_version", "qwm_status_string", "qwm_cache_sizes", "qwm_cache_init",
    "qwm_build_centroids", "qwm_build_centroids_noalloc", "qwm_update_query_stats", "qwm_append_kv", "qwm_attention",
    "qwm_attention_ext", "qwm_reconstruct", "qwm_top1_shift", "qwm_device_status", "QuantKVCache",
    "QWM_FLAG_QSAC_FULL", "QWM_NOALLOC_SCRATCH_BYTES", "QWM_ATTN_MAX_SPLIT",
    "qwm_rope", "qwm_pages", "qwm_rope_init", "qwm_norm_rope", "qwm_paged_append",
    "qwm_attention_shared_workspace", "qwm_attention_shared", "qwm_cross_attention_workspace",
    "qwm_cross_attention", "PagedKV", "ROPE_LAYOUTS", "ROPE_SCALINGS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqwm.so")

QWM_FLAG_QSAC_FULL = 1   # QSAC stage 2 by the full quadratic form e^T A e
QWM_NOALLOC_SCRATCH_BYTES = 16 << 20   # fixed scratch of qwm_build_centroids_noalloc
QWM_ATTN_MAX_SPLIT = 6                 # key ranges an attention call may be split into

BUFFER_NAMES = ["k_codes", "k_params", "k_idx", "k_coef", "k_cscale", "v_codes", "v_params",
                "v_idx", "cent_k", "cent_v", "qstats", "sens", "wgroup", "basis", "tokver",
                "centver", "eigvec", "workspace"]
NBUF = len(BUFFER_NAMES)

STATUS = {0: "QWM_OK", 1: "QWM_ERR_INVALID_ARG", 2: "QWM_ERR_ALIGNMENT", 3: "QWM_ERR_CAPACITY",
          4: "QWM_ERR_STATE", 5: "QWM_ERR_CUDA", 6: "QWM_ERR_TIMEOUT", 7: "QWM_ERR_UNSUPPORTED"}


class qwm_config(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_centroids", ctypes.c_int32), ("group", ctypes.c_int32),
                ("n_cand", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("max_versions", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("max_cent_versions", ctypes.c_int32), ("max_queries", ctypes.c_int32),
                ("max_tokens", ctypes.c_int64)]


class qwm_sizes(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_uint64 * NBUF), ("tcap", ctypes.c_int64),
                ("bytes_per_token_head", ctypes.c_int64)]


class qwm_buffers(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p * NBUF)]


class qwm_cache(ctypes.Structure):
    _fields_ = [("cfg", qwm_config), ("buf", qwm_buffers), ("tcap", ctypes.c_int64),
                ("len", ctypes.c_int64), ("n_queries", ctypes.c_int64),
                ("frames", ctypes.c_int32), ("n_versions", ctypes.c_int32),
                ("cur_version", ctypes.c_int32), ("has_centroids", ctypes.c_int32),
                ("has_eigvec", ctypes.c_int32), ("magic", ctypes.c_int32),
                ("n_cent_versions", ctypes.c_int32), ("cur_cent_version", ctypes.c_int32)]


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


class qwm_rope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("axis_dim", ctypes.c_int32 * 3), ("magic", ctypes.c_int32),
                ("gain", ctypes.c_double), ("freq", ctypes.c_double * 64)]


class qwm_pages(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QwmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")


_lib = None
_P = ctypes.c_void_p


def lib():
    """Load libqwm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libqwm.so not built ({LIB_PATH}); run "
                              "python -m bit_kv_cache_23_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        I32, I64, F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        U64, F64 = ctypes.c_uint64, ctypes.c_double
        pc = ctypes.POINTER(qwm_cache)
        sig = {
            "qwm_abi_version": (I32, []),
            "qwm_status_string": (ctypes.c_char_p, [I32]),
            "qwm_cache_sizes": (I32, [ctypes.POINTER(qwm_config), ctypes.POINTER(qwm_sizes)]),
            "qwm_cache_init": (I32, [pc, ctypes.POINTER(qwm_config), ctypes.POINTER(qwm_buffers), _P]),
            "qwm_build_centroids": (I32, [pc, _P, _P, I64, I32, _P]),
            "qwm_update_query_stats": (I32, [pc, _P, I64, I32, _P]),
            "qwm_append_kv": (I32, [pc, _P, _P, I64, _P]),
            "qwm_attention": (I32, [pc, _P, I64, F32, _P, _P]),
            "qwm_attention_ext": (I32, [pc, _P, I64, _P, _P, I64, F32, _P, _P, _P]),
            "qwm_reconstruct": (I32, [pc, I64, I64, _P, _P, _P]),
            "qwm_top1_shift": (I32, [pc, _P, I64, _P, _P, _P, _P]),
            "qwm_device_status": (I32, [ctypes.POINTER(ctypes.c_int32)]),
            "qwm_build_centroids_noalloc": (I32, [pc, _P, _P, I64, I32, _P]),
            "qwm_rope_init": (I32, [ctypes.POINTER(qwm_rope), I32, I32, I32, F64, I32,
                                    ctypes.POINTER(I32), I32, F64, F64, F64, F64]),
            "qwm_norm_rope": (I32, [_P, I32, I64, _P, I64, I32, _P, _P, I64, _P, I64, I32, _P, _P,
                                    I64, _P, I64, F32, _P]),
            "qwm_paged_append": (I32, [ctypes.POINTER(qwm_pages), _P, I64, I32, _P, _P, _P, I64, _P,
                                       I64, I64, _P, _P, I64, _P, F32, _P]),
            "qwm_attention_shared_workspace": (I32, [pc, I64, I32, I64, I64, I64, _P, _P]),
            "qwm_attention_shared": (I32, [pc, _P, I64, I64, I32, _P, I64, I64, _P, _P, I32, _P, I64,
                                           I32, F32, _P, _P, _P, U64, _P]),
            "qwm_cross_attention_workspace": (I32, [I32, I32, I32, I64, I64, I64, I64, _P, _P]),
            "qwm_cross_attention": (I32, [_P, I64, I64, I32, _P, I64, _P, I64, I64, I32, I32, _P, _P,
                                          _P, I64, I64, I64, F32, _P, _P, _P, U64, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise QwmError(fn, st)


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made(stream, index, make):
    """make(), which allocates, with `stream` (None: the current stream) as the current one.
    Memory of another stream's pool may be free with its last use still queued there, and
    work on `stream` does not wait for that."""
    if stream is None:
        return make()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    with torch.cuda.stream(stream):
        return make()


def _read_here(o, stream, index):
    """o, which a call on `stream` writes and its caller reads on the current stream."""
    if stream is not None:
        o.record_stream(torch.cuda.current_stream(index))
    return o


def _new(x, stream, index):
    """A contiguous tensor like x, an output of a call on `stream`."""
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _read_here(_made(stream, index, lambda: torch.empty_like(x, memory_format=torch.contiguous_format)),
                      stream, index)


def _fresh(shape, dtype, device, stream):
    """A tensor of `shape`, an output of a call on `stream`."""
    return _read_here(_made(stream, device, lambda: torch.empty(shape, dtype=dtype, device=device)), stream, device)


def _dev_ptr(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# ----------------------------------------------------------------- thin entry points
def qwm_abi_version() -> int:
    return int(lib().qwm_abi_version())


def qwm_status_string(status: int) -> str:
    return lib().qwm_status_string(status).decode()


def qwm_cache_sizes(cfg: qwm_config) -> qwm_sizes:
    out = qwm_sizes()
    _check("qwm_cache_sizes", lib().qwm_cache_sizes(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def qwm_cache_init(cache: qwm_cache, cfg: qwm_config, bufs: qwm_buffers, stream=None,
                   device=None) -> None:
    _check("qwm_cache_init", lib().qwm_cache_init(ctypes.byref(cache), ctypes.byref(cfg),
                                                  ctypes.byref(bufs), _stream(stream, device)))


def qwm_build_centroids(cache: qwm_cache, K: torch.Tensor, V: torch.Tensor, iters: int = 10,
                        stream=None) -> None:
    _check("qwm_build_centroids", lib().qwm_build_centroids(
        ctypes.byref(cache), _dev_ptr(K, "K", torch.bfloat16), _dev_ptr(V, "V", torch.bfloat16),
        K.shape[0], iters, _stream(stream, K.device)))


def qwm_build_centroids_noalloc(cache: qwm_cache, K: torch.Tensor, V: torch.Tensor,
                                iters: int = 10, stream=None) -> None:
    """Same result as qwm_build_centroids, with the scratch taken from a fixed
    device array inside the library (for callers that cannot allocate)."""
    _check("qwm_build_centroids_noalloc", lib().qwm_build_centroids_noalloc(
        ctypes.byref(cache), _dev_ptr(K, "K", torch.bfloat16), _dev_ptr(V, "V", torch.bfloat16),
        K.shape[0], iters, _stream(stream, K.device)))


def qwm_update_query_stats(cache: qwm_cache, Q: torch.Tensor, refresh_basis: bool = True,
                           stream=None) -> None:
    _check("qwm_update_query_stats", lib().qwm_update_query_stats(
        ctypes.byref(cache), _dev_ptr(Q, "Q", torch.bfloat16), Q.shape[0], int(refresh_basis),
        _stream(stream, Q.device)))


def qwm_append_kv(cache: qwm_cache, K: torch.Tensor, V: torch.Tensor, stream=None) -> None:
    _check("qwm_append_kv", lib().qwm_append_kv(
        ctypes.byref(cache), _dev_ptr(K, "K", torch.bfloat16), _dev_ptr(V, "V", torch.bfloat16),
        K.shape[0], _stream(stream, K.device)))


def qwm_attention(cache: qwm_cache, Q: torch.Tensor, O: torch.Tensor | None = None,
                  scale: float = 0.0, stream=None) -> torch.Tensor:
    qp = _dev_ptr(Q, "Q", torch.bfloat16)
    if O is None:
        O = _new(Q, stream, Q.get_device())
    _check("qwm_attention", lib().qwm_attention(
        ctypes.byref(cache), qp, Q.shape[0], float(scale),
        _dev_ptr(O, "O", torch.bfloat16), _stream(stream, Q.device)))
    return O


def qwm_attention_ext(cache: qwm_cache, Q: torch.Tensor, K_seg: torch.Tensor | None = None,
                      V_seg: torch.Tensor | None = None, O: torch.Tensor | None = None,
                      lse: torch.Tensor | None = None, scale: float = 0.0,
                      stream=None) -> torch.Tensor:
    """Attention over the packed cache followed by the bf16 segment (K_seg, V_seg),
    [n_seg][H][d]; lse, if given, is a [n_q][H] float32 tensor that receives the
    natural-log softmax denominators."""
    qp = _dev_ptr(Q, "Q", torch.bfloat16)
    if O is None:
        O = _new(Q, stream, Q.get_device())
    n_seg = 0 if K_seg is None else K_seg.shape[0]
    if (K_seg is None) != (V_seg is None) or (V_seg is not None and V_seg.shape != K_seg.shape):
        raise ValueError("K_seg and V_seg must be given together, with equal shapes")
    kp = _dev_ptr(K_seg, "K_seg", torch.bfloat16) if n_seg else None
    vp = _dev_ptr(V_seg, "V_seg", torch.bfloat16) if n_seg else None
    lp = _dev_ptr(lse, "lse", torch.float32) if lse is not None else None
    _check("qwm_attention_ext", lib().qwm_attention_ext(
        ctypes.byref(cache), qp, Q.shape[0], kp, vp, n_seg,
        float(scale), _dev_ptr(O, "O", torch.bfloat16), lp, _stream(stream, Q.device)))
    return O


def qwm_reconstruct(cache: qwm_cache, t0: int, n: int, device, stream=None):
    H, d = cache.cfg.heads, cache.cfg.head_dim
    Kp, Vp = (_fresh((H, n, d), torch.bfloat16, device, stream) for _ in range(2))
    _check("qwm_reconstruct", lib().qwm_reconstruct(
        ctypes.byref(cache), int(t0), int(n), _dev_ptr(Kp, "Kp"), _dev_ptr(Vp, "Vp"),
        _stream(stream, device)))
    return Kp, Vp


def qwm_top1_shift(cache: qwm_cache, Q: torch.Tensor, K_exact: torch.Tensor, stream=None):
    H = cache.cfg.heads
    qp, kp = _dev_ptr(Q, "Q", torch.bfloat16), _dev_ptr(K_exact, "K_exact", torch.bfloat16)
    ie, iq = (_fresh((Q.shape[0], H), torch.int32, Q.device, stream) for _ in range(2))
    _check("qwm_top1_shift", lib().qwm_top1_shift(
        ctypes.byref(cache), qp, Q.shape[0], kp, _dev_ptr(ie, "idx_exact"),
        _dev_ptr(iq, "idx_quant"), _stream(stream, Q.device)))
    return ie, iq


def qwm_device_status() -> int:
    """Synchronize and return 1 if a bounded device wait timed out since the
    last call (the flag is cleared), plus 2 if an offset, length or page number
    in a device array lay outside its buffer and was clamped, else 0."""
    f = ctypes.c_int32(0)
    st = lib().qwm_device_status(ctypes.byref(f))
    if st not in (0, 6) and not (st == 1 and f.value):
        raise QwmError("qwm_device_status", st)
    return int(f.value)


# ----------------------------------------------------------------- around the cache
# These calls are short (a few microseconds on the GPU for single tokens), so a
# tensor that is in order passes one combined test; what is wrong with another is
# found out afterwards.
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _refuse(t, name, index, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)} and strides {t.stride()}, expected {shape}, contiguous")


def _device_of(t, name) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(t, name, None, None, None)
    return t.get_device()


def _rows_ptr(t: torch.Tensor, name: str, index: int, heads=None, dim=None):
    """(pointer, row distance) of a [n][heads][head_dim] bf16 tensor on cuda:index whose
    heads are contiguous within a row; its rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.get_device() != index or t.dim() != 3:
        _refuse(t, name, index, _BF16, "[n][heads][head_dim]")
    n, h, d = t.shape
    if (heads is not None and h != heads) or (dim is not None and d != dim):
        raise ValueError(f"{name} has heads x head_dim = {h} x {d}, expected {heads} x {dim}")
    row, head, one = t.stride()
    if (one != 1 and d > 1) or (head != d and h > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), (row if n > 1 else max(h * d, 8))


def _vec_ptr(t, name, index, dtype, n=None):
    """Pointer of a contiguous vector of n (None: any number) on cuda:index."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or t.dim() != 1
            or (n is not None and t.shape[0] != n) or not t.is_contiguous()):
        _refuse(t, name, index, dtype, f"[{'n' if n is None else n}]")
    return t.data_ptr()


def _mat_ptr(t, name, index, dtype, n=None, m=None):
    """Pointer of a contiguous matrix [n][m] (None: any number) on cuda:index."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or t.dim() != 2
            or (n is not None and t.shape[0] != n) or (m is not None and t.shape[1] != m)
            or not t.is_contiguous()):
        _refuse(t, name, index, dtype, f"[{'n' if n is None else n}][{'m' if m is None else m}]")
    return t.data_ptr()


def _raw_stream(stream, index) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _launch(name: str, index: int, *args) -> None:
    """The library launches on the current device: make it cuda:index for the call."""
    fn = getattr(_lib or lib(), name)
    before = torch._C._cuda_getDevice()
    if before == index:
        st = fn(*args)
    else:
        torch.cuda.set_device(index)
        try:
            st = fn(*args)
        finally:
            torch.cuda.set_device(before)
    if st != 0:
        raise QwmError(name, st)


def qwm_rope_init(head_dim: int, rot_dim: int, layout: str = "half", theta: float = 10000.0,
                  axis_dims=None, scaling: str = "none", factor: float = 1.0,
                  orig_len: float = 4096.0, beta_fast: float = 32.0,
                  beta_slow: float = 1.0) -> qwm_rope:
    """The rotation of `rot_dim` channels: layout "half" or "interleaved", one
    entry of axis_dims per position axis, scaling "none", "linear", "ntk" or
    "parts" (see include/qwm.h)."""
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"layout {layout!r} or scaling {scaling!r} unknown")
    dims = [rot_dim] if axis_dims is None else list(axis_dims)
    r = qwm_rope()
    arr = (ctypes.c_int32 * max(len(dims), 1))(*dims)
    _check("qwm_rope_init", lib().qwm_rope_init(
        ctypes.byref(r), head_dim, rot_dim, ROPE_LAYOUTS[layout], theta, len(dims), arr,
        ROPE_SCALINGS[scaling], factor, orig_len, beta_fast, beta_slow))
    return r


def _pos_ptr(rope, pos, n, index):
    if rope is None:
        if pos is not None:
            raise ValueError("positions without a rotation")
        return None, None
    if pos is None:
        raise ValueError("a rotation needs positions")
    if rope.n_axes == 1 and isinstance(pos, torch.Tensor) and pos.dim() == 1:
        return ctypes.addressof(rope), _vec_ptr(pos, "pos", index, _I32, n)
    return ctypes.addressof(rope), _mat_ptr(pos, "pos", index, _I32, rope.n_axes, n)


def qwm_norm_rope(rope: qwm_rope | None, Q: torch.Tensor | None, K: torch.Tensor | None = None,
                  pos: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                  k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                  Q_out: torch.Tensor | None = None, K_out: torch.Tensor | None = None,
                  stream=None):
    """Per-head RMS norm (where a weight is given) and rotation (where `rope` is)
    of queries and keys in one pass; returns (Q_out, K_out).  Q and K may be
    parts of a fused projection; Q or K may be None.  pos: [axes][n] int32."""
    x0 = Q if Q is not None else K
    if x0 is None:
        raise ValueError("neither Q nor K given")
    index = _device_of(x0, "Q" if Q is not None else "K")
    if Q is not None and K is not None and (Q.shape[0] != K.shape[0] or Q.shape[-1] != K.shape[-1]):
        raise ValueError("Q and K differ in rows or head_dim")
    q, Q_out = _rope_side(Q, q_weight, Q_out, "Q", index, stream)
    k, K_out = _rope_side(K, k_weight, K_out, "K", index, stream)
    n, _, d = x0.shape
    rp, pp = _pos_ptr(rope, pos, n, index)
    _launch("qwm_norm_rope", index, rp, d, n, *q, *k, pp, n, eps, _raw_stream(stream, index))
    return Q_out, K_out


def _rope_side(x, w, o, name, index, stream):
    """One side's arguments of qwm_norm_rope, and its output."""
    if x is None:
        if w is not None or o is not None:
            raise ValueError(f"{name} is missing")
        return (None, 0, 0, None, None, 0), None
    p, ld = _rows_ptr(x, name, index)
    _, h, d = x.shape
    if o is None:
        o = _new(x, stream, index)
        po, ldo = o.data_ptr(), max(h * d, 8)
    else:
        po, ldo = _rows_ptr(o, name + "_out", index)
        if o.shape != x.shape:
            raise ValueError(f"{name}_out must have the shape of {name}")
    return (p, ld, h, None if w is None else _vec_ptr(w, name + " weight", index, _BF16, d), po, ldo), o


def qwm_paged_append(pages: qwm_pages, table: torch.Tensor, cu: torch.Tensor, start: torch.Tensor,
                     K: torch.Tensor, V: torch.Tensor, rope: qwm_rope | None = None,
                     pos: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                     eps: float = 1e-6, stream=None) -> None:
    """Write the rows cu[b] .. cu[b+1]-1 of K (normed and rotated on the way) and
    V to positions start[b], start[b]+1, ... of sequence b's pages."""
    index = _device_of(K, "K")
    kp, ldk = _rows_ptr(K, "K", index, pages.heads, pages.head_dim)
    vp, ldv = _rows_ptr(V, "V", index, pages.heads, pages.head_dim)
    n = K.shape[0]
    if V.shape[0] != n:
        raise ValueError("K and V differ in rows")
    tp = _mat_ptr(table, "table", index, _I32)
    n_seq, width = table.shape
    rp, pp = _pos_ptr(rope, pos, n, index)
    wp = None if k_weight is None else _vec_ptr(k_weight, "k_weight", index, _BF16, pages.head_dim)
    _launch("qwm_paged_append", index, pages, tp, n_seq, width, _vec_ptr(cu, "cu", index, _I32, n_seq + 1),
            _vec_ptr(start, "start", index, _I32, n_seq), kp, ldk, vp, ldv, n, rp, pp, n, wp, eps,
            _raw_stream(stream, index))


def _lse_ptr(lse, n, heads, index):
    return None if lse is None else _mat_ptr(lse, "lse", index, _F32, n, heads)


def _out(O, Q, index, stream):
    if O is None:
        return _new(Q, stream, index)
    if (not isinstance(O, torch.Tensor) or O.dtype is not _BF16 or O.get_device() != index
            or O.shape != Q.shape or not O.is_contiguous()):
        _refuse(O, "O", index, _BF16, f"{tuple(Q.shape)} as Q has")
    return O


def _scratch(workspace, sizes, args, Q, index, stream):
    """(tensor, pointer, bytes): the caller's workspace, or one for this call of the
    full size that sizes(index, *args) gives."""
    if workspace is None:
        nbytes = sizes(index, *args)
        if nbytes == 0:
            return None, None, 0
        workspace = _made(stream, index, lambda: torch.empty(nbytes, dtype=torch.uint8, device=Q.device))
        return workspace, workspace.data_ptr(), nbytes
    if (not isinstance(workspace, torch.Tensor) or workspace.get_device() != index
            or not workspace.is_contiguous()):
        _refuse(workspace, "workspace", index, getattr(workspace, "dtype", None), "any shape")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _full(name, index, args) -> int:
    """The full workspace bytes of a call on cuda:index."""
    if torch._C._cuda_getDevice() == index:
        return _sizes(name, *args)[1]
    with torch.cuda.device(index):
        return _sizes(name, *args)[1]


def _shared_full(index, *args) -> int:
    return _full("qwm_attention_shared_workspace", index, args)


@functools.lru_cache(maxsize=1024)
def _cross_full(index, *args) -> int:   # of the sizes alone, which a program repeats
    return _full("qwm_cross_attention_workspace", index, args)


_TWO = ctypes.c_uint64 * 2


def _sizes(name, *args) -> tuple[int, int]:
    both = _TWO()
    at = ctypes.addressof(both)
    _check(name, getattr(_lib or lib(), name)(*args, at, at + 8))
    return both[0], both[1]


def qwm_attention_shared_workspace(cache: qwm_cache, n_q: int, heads_q: int, n_seq: int, max_q: int,
                                   max_kv: int) -> tuple[int, int]:
    """(least, full) workspace bytes of qwm_attention_shared."""
    return _sizes("qwm_attention_shared_workspace", cache, n_q, heads_q, n_seq, max_q, max_kv)


def qwm_attention_shared(cache: qwm_cache, Q: torch.Tensor, cu: torch.Tensor, max_q: int,
                         pages: qwm_pages | None = None, table: torch.Tensor | None = None,
                         kv_len: torch.Tensor | None = None, max_kv: int | None = None, causal: bool = False,
                         O: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         scale: float = 0.0, workspace: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Attention of the branches (rows cu[b] .. cu[b+1]-1 of Q) over the packed
    history that they share, followed by the first kv_len[b] positions of each
    branch's pages.  max_q, max_kv: upper bounds of a branch's rows and keys, behind
    which they are left out (max_kv None: as many keys as the table has places)."""
    index = _device_of(Q, "Q")
    qp, ldq = _rows_ptr(Q, "Q", index, None, cache.cfg.head_dim)
    n, h, _ = Q.shape
    cup = _vec_ptr(cu, "cu", index, _I32)
    n_seq = cu.shape[0] - 1
    pg = tp = kp = None
    width = 0
    if pages is not None:
        if table is None or kv_len is None:
            raise ValueError("pages need a table and kv_len")
        tp = _mat_ptr(table, "table", index, _I32, n_seq)
        kp = _vec_ptr(kv_len, "kv_len", index, _I32, n_seq)
        pg, width = ctypes.addressof(pages), table.shape[1]
        if max_kv is None:
            max_kv = width * pages.page_size
    elif table is not None or kv_len is not None:
        raise ValueError("a table or kv_len without pages")
    elif max_kv is None:
        max_kv = 0
    O = _out(O, Q, index, stream)
    lp = _lse_ptr(lse, n, h, index)
    ws, wp, wn = _scratch(workspace, _shared_full, (cache, n, h, n_seq, max_q, max_kv), Q,
                          index, stream)
    _launch("qwm_attention_shared", index, cache, qp, ldq, n, h, cup, n_seq, max_q, pg, tp, width, kp,
            max_kv, int(causal), scale, O.data_ptr(), lp, wp, wn, _raw_stream(stream, index))
    return O


def qwm_cross_attention_workspace(heads_q: int, heads_kv: int, head_dim: int, n_q: int, n_seq: int,
                                  max_q: int, max_kv: int) -> tuple[int, int]:
    """(least, full) workspace bytes of qwm_cross_attention."""
    return _sizes("qwm_cross_attention_workspace", heads_q, heads_kv, head_dim, n_q, n_seq, max_q, max_kv)


def qwm_cross_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu: torch.Tensor,
                        kv_start: torch.Tensor, kv_len: torch.Tensor, max_q: int, max_kv: int,
                        O: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        scale: float = 0.0, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Rows cu[b] .. cu[b+1]-1 of Q attend to rows kv_start[b] ..
    kv_start[b]+kv_len[b]-1 of K and V (strided rows allowed)."""
    index = _device_of(Q, "Q")
    qp, ldq = _rows_ptr(Q, "Q", index)
    n, h, d = Q.shape
    kp, ldk = _rows_ptr(K, "K", index, None, d)
    n_kv, hk, _ = K.shape
    vp, ldv = _rows_ptr(V, "V", index, hk, d)
    if V.shape[0] != n_kv:
        raise ValueError("K and V differ in rows")
    cup = _vec_ptr(cu, "cu", index, _I32)
    n_seq = cu.shape[0] - 1
    sp = _vec_ptr(kv_start, "kv_start", index, _I32, n_seq)
    lnp = _vec_ptr(kv_len, "kv_len", index, _I32, n_seq)
    O = _out(O, Q, index, stream)
    lp = _lse_ptr(lse, n, h, index)
    ws, wp, wn = _scratch(workspace, _cross_full, (h, hk, d, n, n_seq, max_q, max_kv), Q,
                          index, stream)
    _launch("qwm_cross_attention", index, qp, ldq, n, h, kp, ldk, vp, ldv, n_kv, hk, d, cup, sp, lnp, n_seq,
            max_q, max_kv, scale, O.data_ptr(), lp, wp, wn, _raw_stream(stream, index))
    return O


class PagedKV:
    """A pool of pages of bf16 keys and values, [n_pages][heads][page_size][head_dim]
    each; the pools are the caller's tensors (PagedKV.empty allocates them)."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor):
        if K.dim() != 4 or K.shape != V.shape or K.device != V.device:
            raise ValueError("K and V must be [n_pages][heads][page_size][head_dim] alike")
        self.K, self.V = K, V
        n, h, p, d = K.shape
        self.pages = qwm_pages(_dev_ptr(K, "K", torch.bfloat16).value,
                               _dev_ptr(V, "V", torch.bfloat16).value, n, h, d, p, 0)

    @classmethod
    def empty(cls, n_pages: int, heads: int, page_size: int, head_dim: int, device="cuda"):
        shape = (n_pages, heads, page_size, head_dim)
        return cls(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))

    def append(self, table, cu, start, K, V, rope=None, pos=None, k_weight=None, eps=1e-6,
               stream=None):
        if K.device != self.K.device:
            raise ValueError(f"K is on {K.device}, the pages on {self.K.device}")
        qwm_paged_append(self.pages, table, cu, start, K, V, rope, pos, k_weight, eps, stream)


# ----------------------------------------------------------------- convenience owner
class QuantKVCache:
    """Allocates the caller-owned device buffers with torch and holds the host
    state; every method is one C-ABI call."""

    def __init__(self, heads: int, head_dim: int, n_centroids: int, group: int, n_cand: int,
                 rank: int, max_tokens: int, max_versions: int = 1024, device="cuda",
                 stream=None, qsac_full: bool = False, max_cent_versions: int = 1,
                 max_queries: int = 0):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("QuantKVCache lives on a CUDA device")
        flags = QWM_FLAG_QSAC_FULL if qsac_full else 0
        self.cfg = qwm_config(heads, head_dim, n_centroids, group, n_cand, rank, max_versions,
                              flags, max_cent_versions, max_queries, max_tokens)
        self.sizes = qwm_cache_sizes(self.cfg)
        self.buffers = {}
        bufs = qwm_buffers()
        for i, name in enumerate(BUFFER_NAMES):
            nb = int(self.sizes.bytes[i])
            t = _fresh((max(nb, 256),), torch.uint8, self.device, stream)
            self.buffers[name] = t
            bufs.ptr[i] = t.data_ptr()
        self.bufs = bufs
        self.c = qwm_cache()
        qwm_cache_init(self.c, self.cfg, bufs, stream, self.device)

    # host state
    @property
    def len(self) -> int:
        return int(self.c.len)

    @property
    def tcap(self) -> int:
        return int(self.sizes.tcap)

    @property
    def version(self) -> int:
        return int(self.c.cur_version)

    @property
    def cent_version(self) -> int:
        return int(self.c.cur_cent_version)

    def build_centroids(self, K, V, iters=10, stream=None):
        qwm_build_centroids(self.c, K, V, iters, stream)

    def update_query_stats(self, Q, refresh_basis=True, stream=None):
        qwm_update_query_stats(self.c, Q, refresh_basis, stream)

    def append_kv(self, K, V, stream=None):
        qwm_append_kv(self.c, K, V, stream)

    def attention(self, Q, O=None, scale=0.0, stream=None):
        return qwm_attention(self.c, Q, O, scale, stream)

    def attention_ext(self, Q, K_seg=None, V_seg=None, O=None, lse=None, scale=0.0,
                      stream=None):
        return qwm_attention_ext(self.c, Q, K_seg, V_seg, O, lse, scale, stream)

    def attention_shared(self, Q, cu, max_q, pages: PagedKV | None = None, table=None, kv_len=None,
                         max_kv=None, causal=False, O=None, lse=None, scale=0.0, workspace=None,
                         stream=None):
        if Q.device != self.buffers["k_codes"].device:
            raise ValueError(f"Q is on {Q.device}, the cache on {self.device}")
        if pages is not None and pages.K.device != Q.device:
            raise ValueError(f"Q is on {Q.device}, the pages on {pages.K.device}")
        return qwm_attention_shared(self.c, Q, cu, max_q, pages.pages if pages else None, table,
                                    kv_len, max_kv, causal, O, lse, scale, workspace, stream)

    def reconstruct(self, t0=0, n=None, stream=None):
        n = self.len - t0 if n is None else n
        return qwm_reconstruct(self.c, t0, n, self.device, stream)

    def top1_shift(self, Q, K_exact, stream=None):
        return qwm_top1_shift(self.c, Q, K_exact, stream)

    # typed views of the packed buffers (for inspection and tests); the centroid
    # tables are those of `cent_version` (default: the version in force)
    def view(self, name: str, cent_version: int | None = None) -> torch.Tensor:
        H, d, C, G, r = (self.cfg.heads, self.cfg.head_dim, self.cfg.n_centroids,
                         self.cfg.group, self.cfg.rank)
        if name in ("cent_k", "cent_v"):
            cv = self.cent_version if cent_version is None else int(cent_version)
            if not 0 <= cv < self.cfg.max_cent_versions:
                raise IndexError(f"centroid-table version {cv} out of range")
            n = H * C * d
            return self.buffers[name][2 * n * cv:2 * n * (cv + 1)].view(torch.int16).view(H, C, d)
        T, ng = self.tcap, d // G
        b = self.buffers[name]
        idt = torch.uint8 if C <= 256 else torch.int16
        shapes = {
            "k_codes": (torch.uint8, (H, T, d // 4)), "v_codes": (torch.uint8, (H, T, d // 4)),
            "k_params": (torch.int16, (H, T, ng, 2)), "v_params": (torch.int16, (H, T, ng, 2)),
            "k_idx": (idt, (H, T)), "v_idx": (idt, (H, T)),
            "k_coef": (torch.int8, (H, T, r)), "k_cscale": (torch.int16, (H, T)),
            "qstats": (torch.float64, (H, d, d)), "sens": (torch.float32, (H, d)),
            "wgroup": (torch.float32, (H, ng)), "tokver": (torch.int16, (T,)),
            "centver": (torch.int16, (T,)),
            "basis": (torch.float32, (self.cfg.max_versions, H, d, max(r, 1))),
            "eigvec": (torch.float64, (H * d * d + H,)),
        }
        dt, shp = shapes[name]
        n = math.prod(shp) * torch.empty((), dtype=dt).element_size()
        return b[:n].view(dt).view(shp)
