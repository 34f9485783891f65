"""Thin Python binding of librq.so (include/rq.h).

Argument marshalling only: every step of quantize-append and attention runs in the CUDA
kernels of librq.so.  PyTorch tensors supply device memory and the current CUDA stream.
There is no CPU fallback: if the library cannot be built or loaded, every call raises.

Low-level functions carry the C names (rq_create, rq_quantize_append, rq_decode_attention,
rq_verify_attention, rq_free, ...); `KVCache` bundles a context with its page pool.
"""
from __future__ import annotations

import ctypes
import threading

import numpy as np
import torch

from . import build as _build

RQ_OK, RQ_ERR_INVALID, RQ_ERR_UNSUPPORTED, RQ_ERR_CUDA, RQ_ERR_CAPACITY = 0, 1, 2, 3, 4
RQ_STATUS_BAD_PAGE, RQ_STATUS_BAD_SLOT, RQ_STATUS_BAD_LEN, RQ_STATUS_NORM_OVERFLOW, RQ_STATUS_TIMEOUT = 1, 2, 4, 8, 16
RQ_STATUS_NOT_FINITE, RQ_STATUS_BAD_ORDER = 32, 64
RQ_PLANAR, RQ_ISO, RQ_DENSE = 0, 1, 2
RQ_FP8 = 8
RQ_F16, RQ_BF16 = 0, 1
HEAD_DIM = 128
BLOCK_TOKENS, BLOCK_BYTES = 16, 4112  # RQ_FP8: tokens that share a scale, bytes of such a block
_IO_TYPES = {torch.float16: RQ_F16, torch.bfloat16: RQ_BF16}

EXPORTS = ["rq_create", "rq_free", "rq_page_bytes", "rq_lloyd_max_codebook", "rq_get_codebook",
           "rq_quantize_append", "rq_decode_attention", "rq_verify_attention", "rq_set_profile_events",
           "rq_decode_attention_noalloc", "rq_tree_verify_attention", "rq_decode_step", "rq_extend_attention", "rq_status_string",
           "rq_rope_create", "rq_rope_free", "rq_norm_rope", "rq_rope_append"]


class RQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {status_string(code)} ({code})")
        self.code = code


class rq_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int), ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
        ("bits", ctypes.c_int), ("mode", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("max_batch", ctypes.c_int), ("max_query_tokens", ctypes.c_int), ("max_pages_per_seq", ctypes.c_int),
        ("rot_k", ctypes.POINTER(ctypes.c_float)), ("rot_v", ctypes.POINTER(ctypes.c_float)),
        ("codebook", ctypes.POINTER(ctypes.c_float)), ("sm_scale", ctypes.c_float), ("device", ctypes.c_int),
        ("io_type", ctypes.c_int),
    ]


class rq_rope_config(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("num_axes", ctypes.c_int),
        ("inv_freq", ctypes.POINTER(ctypes.c_double)), ("axis", ctypes.POINTER(ctypes.c_int)),
        ("scale", ctypes.c_float), ("device", ctypes.c_int),
    ]


class rq_rows(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("stride", ctypes.c_longlong), ("heads", ctypes.c_int), ("weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("out_stride", ctypes.c_longlong),
    ]


class Context(ctypes.c_void_p):
    """An rq_ctx and the element type of its q, k, v and out."""
    dtype = torch.float16


_lock = threading.Lock()
_lib = None


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load librq.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None and path is None:  # loaded: no lock on the call path
        return _lib
    with _lock:
        if _lib is None:
            L = ctypes.CDLL(path or _build.build())
            vp, i32p, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_float)
            L.rq_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(rq_config)]
            L.rq_create.restype = ctypes.c_int
            L.rq_free.argtypes = [vp]
            L.rq_free.restype = None
            L.rq_page_bytes.argtypes = [vp]
            L.rq_page_bytes.restype = ctypes.c_size_t
            L.rq_lloyd_max_codebook.argtypes = [ctypes.c_int, ctypes.c_int, fp]
            L.rq_lloyd_max_codebook.restype = ctypes.c_int
            L.rq_get_codebook.argtypes = [vp, fp, fp]
            L.rq_get_codebook.restype = ctypes.c_int
            L.rq_quantize_append.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, vp, vp]
            L.rq_quantize_append.restype = ctypes.c_int
            L.rq_decode_attention.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp]
            L.rq_decode_attention.restype = ctypes.c_int
            L.rq_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp]
            L.rq_decode_step.restype = ctypes.c_int
            L.rq_extend_attention.argtypes = [vp, vp, ctypes.c_int, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp]
            L.rq_extend_attention.restype = ctypes.c_int
            L.rq_verify_attention.argtypes = [vp, vp, ctypes.c_int, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp,
                                              vp]
            L.rq_verify_attention.restype = ctypes.c_int
            L.rq_tree_verify_attention.argtypes = [vp, vp, ctypes.c_int, vp, vp, vp, ctypes.c_int, vp, ctypes.c_int,
                                                   vp, vp, vp]
            L.rq_tree_verify_attention.restype = ctypes.c_int
            L.rq_decode_attention_noalloc.argtypes = [ctypes.POINTER(rq_config), vp, vp, vp, vp, vp, vp,
                                                      ctypes.c_int, vp, ctypes.c_int, vp, vp, vp]
            L.rq_decode_attention_noalloc.restype = ctypes.c_int
            L.rq_set_profile_events.argtypes = [vp, vp, vp]
            L.rq_set_profile_events.restype = ctypes.c_int
            rows = ctypes.POINTER(rq_rows)
            L.rq_rope_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(rq_rope_config)]
            L.rq_rope_create.restype = ctypes.c_int
            L.rq_rope_free.argtypes = [vp]
            L.rq_rope_free.restype = None
            L.rq_norm_rope.argtypes = [vp, rows, rows, ctypes.c_int, ctypes.c_float, vp, ctypes.c_int, vp]
            L.rq_norm_rope.restype = ctypes.c_int
            L.rq_rope_append.argtypes = [vp, vp, rows, rows, vp, ctypes.c_longlong, ctypes.c_float, vp, vp,
                                         ctypes.c_int, vp, vp, vp]
            L.rq_rope_append.restype = ctypes.c_int
            L.rq_status_string.argtypes = [ctypes.c_int]
            L.rq_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().rq_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != RQ_OK:
        raise RQError(fn, code)


def _ptr(t):
    """An address for a c_void_p argument (ctypes converts the int itself)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return int(t)


def _dtype(ctx):
    """The element type that a context's q, k, v and out have."""
    return getattr(ctx, "dtype", torch.float16)


def _stream(stream, device) -> int:
    if stream is None:  # the handle alone: a Stream object costs 2 us a call
        index = device.index
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def rq_lloyd_max_codebook(bits: int, head_dim: int = HEAD_DIM) -> np.ndarray:
    out = np.zeros(1 << bits, np.float32)
    _check("rq_lloyd_max_codebook",
           lib().rq_lloyd_max_codebook(bits, head_dim, out.ctypes.data_as(ctypes.POINTER(ctypes.c_float))))
    return out


def rq_create(mode: int, bits: int, num_q_heads: int, num_kv_heads: int, page_size: int, num_pages: int,
              rot_k, rot_v, max_batch: int, max_query_tokens: int = 1, max_pages_per_seq: int = 1,
              codebook=None, sm_scale: float = 0.0, device: int = -1, dtype=torch.float16) -> ctypes.c_void_p:
    """rot_k, rot_v: None for RQ_FP8.  dtype: the element type of q, k, v and out (bfloat16: RQ_FP8 only)."""
    fp = ctypes.POINTER(ctypes.c_float)
    ctx = Context()
    if dtype not in _IO_TYPES:
        raise RQError("rq_create", RQ_ERR_UNSUPPORTED)
    ctx.dtype = dtype
    if mode == RQ_FP8:
        if rot_k is not None or rot_v is not None or codebook is not None:
            raise RQError("rq_create", RQ_ERR_INVALID)
        cfg = rq_config(HEAD_DIM, num_q_heads, num_kv_heads, bits, mode, page_size, num_pages, max_batch,
                        max_query_tokens, max_pages_per_seq, fp(), fp(), fp(), float(sm_scale), int(device),
                        _IO_TYPES[dtype])
        _check("rq_create", lib().rq_create(ctypes.byref(ctx), ctypes.byref(cfg)))
        return ctx
    rk = np.ascontiguousarray(rot_k, np.float32).reshape(-1)
    rv = np.ascontiguousarray(rot_v, np.float32).reshape(-1)
    want = num_kv_heads * HEAD_DIM * (HEAD_DIM if mode == RQ_DENSE else 1)
    if rk.size != want or rv.size != want:  # the library reads exactly `want` floats of each
        raise RQError("rq_create", RQ_ERR_INVALID)
    cb = None if codebook is None else np.ascontiguousarray(codebook, np.float32)
    cfg = rq_config(HEAD_DIM, num_q_heads, num_kv_heads, bits, mode, page_size, num_pages, max_batch,
                    max_query_tokens, max_pages_per_seq, rk.ctypes.data_as(fp), rv.ctypes.data_as(fp),
                    cb.ctypes.data_as(fp) if cb is not None else fp(), float(sm_scale), int(device), _IO_TYPES[dtype])
    _check("rq_create", lib().rq_create(ctypes.byref(ctx), ctypes.byref(cfg)))
    return ctx


def rq_free(ctx) -> None:
    lib().rq_free(ctx)


def rq_page_bytes(ctx) -> int:
    return int(lib().rq_page_bytes(ctx))


def rq_get_codebook(ctx, bits: int):
    c = np.zeros(1 << bits, np.float32)
    b = np.zeros((1 << bits) - 1, np.float32)
    fp = ctypes.POINTER(ctypes.c_float)
    _check("rq_get_codebook", lib().rq_get_codebook(ctx, c.ctypes.data_as(fp), b.ctypes.data_as(fp)))
    return c, b


def rq_quantize_append(ctx, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, kv_pages: torch.Tensor,
                       status: torch.Tensor | None = None, stream=None) -> None:
    """k, v: fp16 [n][Hkv][128] on the device; slot_mapping int32 [n]."""
    n = slot_mapping.numel()
    if n:
        assert k.dtype == _dtype(ctx) and v.dtype == _dtype(ctx) and slot_mapping.dtype == torch.int32
        assert k.is_contiguous() and v.is_contiguous() and slot_mapping.is_contiguous()
    _check("rq_quantize_append",
           lib().rq_quantize_append(ctx, _ptr(k), _ptr(v), _ptr(slot_mapping), n, _ptr(kv_pages), _ptr(status),
                                    _stream(stream, kv_pages.device)))


def rq_decode_attention(ctx, q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, out: torch.Tensor, status: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """q, out: fp16 [B][Hq][128]; block_table int32 [B][max_pages]; seq_lens int32 [B]."""
    B = seq_lens.numel()
    assert q.dtype == _dtype(ctx) and out.dtype == _dtype(ctx) and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    _check("rq_decode_attention",
           lib().rq_decode_attention(ctx, _ptr(q), _ptr(kv_pages), _ptr(block_table), block_table.shape[-1],
                                     _ptr(seq_lens), B, _ptr(out), _ptr(status), _stream(stream, q.device)))
    return out


def rq_decode_step(ctx, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, kv_pages: torch.Tensor,
                   block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                   status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step: append k_new / v_new (fp16 [B][Hkv][128]) at position seq_lens[b] - 1 of
    each sequence, then decode attention; q, out fp16 [B][Hq][128]."""
    B = seq_lens.numel()
    for t in (q, out, k_new, v_new):
        assert t.dtype == _dtype(ctx) and t.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    _check("rq_decode_step",
           lib().rq_decode_step(ctx, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kv_pages), _ptr(block_table),
                                block_table.shape[-1], _ptr(seq_lens), B, _ptr(out), _ptr(status),
                                _stream(stream, q.device)))
    return out


def rq_extend_attention(ctx, q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, out: torch.Tensor, status: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Extend (prefill) attention: q, out fp16 [B][T][Hq][128]; row j sees positions <= len - T + j."""
    B, T = q.shape[0], q.shape[1]
    assert q.dtype == _dtype(ctx) and out.dtype == _dtype(ctx) and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    _check("rq_extend_attention",
           lib().rq_extend_attention(ctx, _ptr(q), T, _ptr(kv_pages), _ptr(block_table), block_table.shape[-1],
                                     _ptr(seq_lens), B, _ptr(out), _ptr(status), _stream(stream, q.device)))
    return out


def rq_verify_attention(ctx, q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                        seq_lens: torch.Tensor, out: torch.Tensor, status: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """q, out: fp16 [B][T][Hq][128]."""
    B, T = q.shape[0], q.shape[1]
    assert q.dtype == _dtype(ctx) and out.dtype == _dtype(ctx) and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    _check("rq_verify_attention",
           lib().rq_verify_attention(ctx, _ptr(q), T, _ptr(kv_pages), _ptr(block_table), block_table.shape[-1],
                                     _ptr(seq_lens), B, _ptr(out), _ptr(status), _stream(stream, q.device)))
    return out


def rq_tree_verify_attention(ctx, q: torch.Tensor, tree_mask: torch.Tensor, kv_pages: torch.Tensor,
                             block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                             status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q, out: fp16 [B][T][Hq][128]; tree_mask int64/uint64 [B][T] (bit i of row j: draft i visible)."""
    B, T = q.shape[0], q.shape[1]
    assert q.dtype == _dtype(ctx) and out.dtype == _dtype(ctx) and q.is_contiguous() and out.is_contiguous()
    assert tree_mask.dtype in (torch.int64, torch.uint64) and tree_mask.is_contiguous() and tuple(tree_mask.shape) == (B, T)
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    _check("rq_tree_verify_attention",
           lib().rq_tree_verify_attention(ctx, _ptr(q), T, _ptr(tree_mask), _ptr(kv_pages), _ptr(block_table),
                                          block_table.shape[-1], _ptr(seq_lens), B, _ptr(out), _ptr(status),
                                          _stream(stream, q.device)))
    return out


def rq_decode_attention_noalloc(mode: int, bits: int, num_q_heads: int, num_kv_heads: int, page_size: int,
                                num_pages: int, d_rot_k: torch.Tensor, d_rot_v: torch.Tensor,
                                d_centroids: torch.Tensor, q: torch.Tensor, kv_pages: torch.Tensor,
                                block_table: torch.Tensor, seq_lens: torch.Tensor, out: torch.Tensor,
                                status: torch.Tensor | None = None, sm_scale: float = 0.0,
                                stream=None) -> torch.Tensor:
    """Decode attention with no allocation: tables as device float32 tensors, scratch in the
    library's fixed device array (see include/rq.h)."""
    for t in (d_rot_k, d_rot_v, d_centroids):
        assert t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda
    assert q.dtype == torch.float16 and out.dtype == torch.float16 and q.is_contiguous() and out.is_contiguous()
    assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32 and block_table.is_contiguous()
    cfg = rq_config(HEAD_DIM, num_q_heads, num_kv_heads, bits, mode, page_size, num_pages, 0, 0, 0,
                    ctypes.POINTER(ctypes.c_float)(), ctypes.POINTER(ctypes.c_float)(),
                    ctypes.POINTER(ctypes.c_float)(), float(sm_scale), -1)
    _check("rq_decode_attention_noalloc",
           lib().rq_decode_attention_noalloc(ctypes.byref(cfg), _ptr(d_rot_k), _ptr(d_rot_v), _ptr(d_centroids),
                                             _ptr(q), _ptr(kv_pages), _ptr(block_table), block_table.shape[-1],
                                             _ptr(seq_lens), seq_lens.numel(), _ptr(out), _ptr(status),
                                             _stream(stream, q.device)))
    return out


def _rows(t, name: str, weight=None, out=None) -> rq_rows:
    """rq_rows of t [n][heads][128] (heads and dims contiguous, any stride from token to token)."""
    shape, stride = t.shape, t.stride()
    heads = shape[1] if len(shape) == 3 else 0
    least = heads * HEAD_DIM
    # the stride of a single token says nothing
    st, out_st, out_ptr = stride[0] if shape[0] > 1 else least, 0, None
    ok = heads > 0 and shape[2] == HEAD_DIM and stride[2] == 1 and (stride[1] == HEAD_DIM or heads == 1)
    if out is not None:
        o = out.stride()
        ok = ok and out.shape == shape and out.dtype == t.dtype and out.device == t.device
        ok = ok and o[2] == 1 and (o[1] == HEAD_DIM or heads == 1)
        out_st, out_ptr = o[0] if shape[0] > 1 else least, out.data_ptr()
    wptr = None
    if weight is not None:
        ok = (ok and weight.dtype == torch.float32 and weight.shape == (HEAD_DIM,) and weight.is_contiguous() and
              weight.device == t.device)
        wptr = weight.data_ptr()
    if not ok:
        raise RQError(name, RQ_ERR_INVALID)
    return rq_rows(t.data_ptr(), st, heads, wptr, out_ptr, out_st)


def _positions(positions, n: int, axes: int, device, name: str):
    """int32 [axes][n] (one axis: also [n])."""
    if axes == 0:
        return None
    if (positions is None or positions.dtype != torch.int32 or positions.device != device or
            not positions.is_contiguous() or
            (positions.shape != (axes, n) and (axes > 1 or positions.shape != (n,)))):
        raise RQError(name, RQ_ERR_INVALID)
    return positions


def rq_rope_create(rotary_dim: int, inv_freq, axis=None, num_axes: int = 1, interleaved: bool = False,
                   scale: float = 0.0, device: int = -1) -> ctypes.c_void_p:
    """inv_freq: float64 [rotary_dim / 2], radians per position; axis: the position axis of each pair."""
    f = np.ascontiguousarray(inv_freq, np.float64).reshape(-1)
    ax = None if axis is None else np.ascontiguousarray(axis, np.intc).reshape(-1)
    if f.size * 2 != rotary_dim or (ax is not None and ax.size != f.size):
        raise RQError("rq_rope_create", RQ_ERR_INVALID)
    cfg = rq_rope_config(rotary_dim, int(interleaved), num_axes, f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                         ax.ctypes.data_as(ctypes.POINTER(ctypes.c_int)) if ax is not None else None, float(scale),
                         int(device))
    rope = ctypes.c_void_p()
    _check("rq_rope_create", lib().rq_rope_create(ctypes.byref(rope), ctypes.byref(cfg)))
    return rope


def rq_rope_free(rope) -> None:
    lib().rq_rope_free(rope)


def rq_norm_rope(rope, q, k, positions, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
                 stream=None) -> None:
    """Norm (where a weight, float32 [128], is given) and rotation (rope None: none) of q, k: fp16 or
    bf16 [n][heads][128] into q_out, k_out; q or k may be None.  The low-level call: positions and
    shapes are checked by Rope.apply."""
    t = q if q is not None else k
    rows = [None if x is None else _rows(x, "rq_norm_rope", w, o) for x, w, o in ((q, q_weight, q_out), (k, k_weight, k_out))]
    _check("rq_norm_rope",
           lib().rq_norm_rope(rope, rows[0], rows[1], _IO_TYPES[t.dtype], float(eps), _ptr(positions), t.shape[0],
                              _stream(stream, t.device)))


def rq_rope_append(ctx, rope, q, k, v, positions, slot_mapping, kv_pages, q_weight=None, k_weight=None,
                   eps: float = 1e-6, q_out=None, status=None, stream=None) -> None:
    """rq_norm_rope of q (into q_out) and k, and the append of k and v, in one launch."""
    rows = [None if q is None else _rows(q, "rq_rope_append", q_weight, q_out), _rows(k, "rq_rope_append", k_weight),
            _rows(v, "rq_rope_append")]
    _check("rq_rope_append",
           lib().rq_rope_append(ctx, rope, rows[0], rows[1], rows[2].x, rows[2].stride, float(eps), _ptr(positions),
                                _ptr(slot_mapping), slot_mapping.numel(), _ptr(kv_pages), _ptr(status),
                                _stream(stream, kv_pages.device)))


def rq_set_profile_events(ctx, ev_start=None, ev_end=None) -> None:
    """Record torch.cuda.Event pairs around the split-K attention kernel of later calls."""
    a = ctypes.c_void_p(ev_start.cuda_event) if ev_start is not None else None
    b = ctypes.c_void_p(ev_end.cuda_event) if ev_end is not None else None
    _check("rq_set_profile_events", lib().rq_set_profile_events(ctx, a, b))


class Rope:
    """Position rotation of query and key heads, with their norms in the same pass.

    rotary_dim: the dims that turn (a multiple of 8, at most 128).  Frequencies (radians per position
    of pair i): inv_freq, or base ** (-2 i / rotary_dim).  interleaved: pairs (2i, 2i + 1) instead of
    (i, i + rotary_dim / 2).  Several position axes (time, height, width): sections, the number of
    consecutive pairs that each axis turns, or axis, the axis of each pair.  scale multiplies cos and
    sin.  Angles are exact at every int32 position."""

    def __init__(self, rotary_dim=HEAD_DIM, base=10000.0, inv_freq=None, sections=None, axis=None, interleaved=False,
                 scale=1.0, device="cuda"):
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.rope = None
        pairs = rotary_dim // 2
        if inv_freq is None:
            inv_freq = base ** (-2.0 * np.arange(pairs, dtype=np.float64) / max(rotary_dim, 1))
        if sections is not None:
            if axis is not None or sum(sections) != pairs or min(sections, default=-1) < 0:
                raise RQError("rq_rope_create", RQ_ERR_INVALID)
            axis = np.repeat(np.arange(len(sections)), sections)
        self.num_axes = len(sections) if sections is not None else 1 if axis is None else int(np.max(axis, initial=0)) + 1
        self.rotary_dim = rotary_dim
        if not scale > 0:
            raise RQError("rq_rope_create", RQ_ERR_INVALID)
        self.rope = rq_rope_create(rotary_dim, inv_freq, axis, self.num_axes, interleaved, scale, self.device.index)

    def positions(self, positions, n, name):
        """positions checked: int32 [n], or [num_axes][n]."""
        return _positions(positions, n, self.num_axes if self.rotary_dim else 0, self.device, name)

    def apply(self, q, k, positions, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
        """(q, k) normed (where a weight, float32 [128], is given) and turned.  q, k: fp16 or bf16
        [n][heads][128], either None; slices of a fused projection's output are taken as they are.
        q_out, k_out: where to write (q, k themselves: in place); new tensors by default."""
        given = [t for t in (q, k) if t is not None]
        first = given[0] if given else None
        if first is None or first.dtype not in _IO_TYPES or first.dim() != 3 or first.device != self.device:
            raise RQError("rq_norm_rope", RQ_ERR_INVALID)
        n = first.shape[0]
        if len(given) == 2 and (k.dtype != first.dtype or k.dim() != 3 or k.shape[0] != n or k.device != self.device):
            raise RQError("rq_norm_rope", RQ_ERR_INVALID)
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        rq_norm_rope(self.rope, q, k, self.positions(positions, n, "rq_norm_rope"), q_weight, k_weight, eps, q_out,
                     k_out, stream)
        return q_out, k_out

    def close(self):
        if self.rope is not None:
            torch.cuda.synchronize(self.device)
            rq_rope_free(self.rope)
            self.rope = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """A context plus its device page pool ([num_pages][Hkv][page_bytes] uint8) and status word.

    mode RQ_FP8 (bits 8, rot_k and rot_v None) holds e4m3 codes with a scale for each block of 16
    tokens and kv head; its q, k, v and outputs have `dtype`, fp16 or bf16 (other modes: fp16).
    pages: a pool of the caller's instead of a new one of zeros."""

    def __init__(self, mode, bits, num_q_heads, num_kv_heads, page_size, num_pages, rot_k, rot_v, max_batch,
                 max_query_tokens=1, max_pages_per_seq=None, codebook=None, sm_scale=0.0, device="cuda",
                 dtype=torch.float16, pages=None):
        self.ctx = None
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.mode, self.bits = mode, bits
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.page_size, self.num_pages = page_size, num_pages
        if max_pages_per_seq is None:
            max_pages_per_seq = num_pages
        self.ctx = rq_create(mode, bits, num_q_heads, num_kv_heads, page_size, num_pages, rot_k, rot_v, max_batch,
                             max_query_tokens, max_pages_per_seq, codebook, sm_scale, self.device.index, dtype)
        self.page_bytes = rq_page_bytes(self.ctx)
        shape = (num_pages, num_kv_heads, self.page_bytes)
        if pages is None:
            pages = torch.zeros(shape, dtype=torch.uint8, device=self.device)
        elif (tuple(pages.shape) != shape or pages.dtype != torch.uint8 or pages.device != self.device or
              not pages.is_contiguous()):
            raise RQError("rq_create", RQ_ERR_INVALID)
        self.pages = pages
        self._views = None
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def codebook(self):
        return rq_get_codebook(self.ctx, self.bits)

    def append(self, k, v, slot_mapping, stream=None):
        rq_quantize_append(self.ctx, k, v, slot_mapping, self.pages, self.status, stream)

    def append_rope(self, k, v, slot_mapping, rope, positions, q=None, q_weight=None, k_weight=None, eps=1e-6,
                    q_out=None, stream=None):
        """RQ_FP8: everything between the projections and attention in one launch -- the norms (where
        a weight is given) and rotation (rope: a Rope, or None) of k on its way into the cache, v
        beside it, and of q, whose result is returned (None without q).  q, k, v: [n][heads][128],
        slices of a fused projection's output are taken as they are; slot_mapping int32 [n]."""
        name, n, device, dtype = "rq_rope_append", slot_mapping.numel(), self.device, _dtype(self.ctx)
        shape = (n, self.num_kv_heads, HEAD_DIM)
        if (k is None or v is None or slot_mapping.dtype != torch.int32 or not slot_mapping.is_contiguous() or
                slot_mapping.device != device or (rope is not None and rope.device != device) or
                k.shape != shape or k.dtype != dtype or k.device != device or
                v.shape != shape or v.dtype != dtype or v.device != device or
                (q is not None and (q.dim() != 3 or q.shape[0] != n or q.dtype != dtype or q.device != device))):
            raise RQError(name, RQ_ERR_INVALID)
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        positions = rope.positions(positions, n, name) if rope is not None else None
        rq_rope_append(self.ctx, rope.rope if rope is not None else None, q, k, v, positions, slot_mapping, self.pages,
                       q_weight, k_weight, eps, q_out, self.status, stream)
        return q_out

    def codes(self):
        """RQ_FP8: the pool's codes as float8_e4m3fn [num_pages][Hkv][page_size / 16][4096] (a view), each
        block's 2048 key codes, then its value codes, in the byte order of include/rq.h."""
        return self._block_views()[0]

    def scales(self):
        """RQ_FP8: the key and value scale of each block, float8_e8m0fnu [num_pages][Hkv][page_size / 16][2] (a view)."""
        return self._block_views()[1]

    def _block_views(self):
        if self.mode != RQ_FP8:
            raise RQError("codes", RQ_ERR_UNSUPPORTED)
        if self._views is None or self._views[2] is not self.pages:
            blocks = self.pages.view(self.num_pages, self.num_kv_heads, self.page_size // BLOCK_TOKENS, BLOCK_BYTES)
            at = 2 * BLOCK_TOKENS * HEAD_DIM
            self._views = (blocks[..., :at].view(torch.float8_e4m3fn),
                           blocks[..., at:at + 2].view(torch.float8_e8m0fnu), self.pages)
        return self._views[:2]

    def decode(self, q, block_table, seq_lens, out=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        return rq_decode_attention(self.ctx, q, self.pages, block_table, seq_lens, out, self.status, stream)

    def decode_step(self, q, k_new, v_new, block_table, seq_lens, out=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        return rq_decode_step(self.ctx, q, k_new, v_new, self.pages, block_table, seq_lens, out, self.status, stream)

    def extend(self, q, block_table, seq_lens, out=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        return rq_extend_attention(self.ctx, q, self.pages, block_table, seq_lens, out, self.status, stream)

    def verify(self, q, block_table, seq_lens, out=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        return rq_verify_attention(self.ctx, q, self.pages, block_table, seq_lens, out, self.status, stream)

    def tree_verify(self, q, tree_mask, block_table, seq_lens, out=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        return rq_tree_verify_attention(self.ctx, q, tree_mask, self.pages, block_table, seq_lens, out, self.status,
                                        stream)

    def close(self):
        if self.ctx is not None:
            torch.cuda.synchronize(self.device)
            rq_free(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
