"""Python binding of libattn.so (the C ABI in include/attn.h).

Argument marshalling only: every step of the attention pass runs in the CUDA
library. Tensors must be CUDA fp16 tensors (uint32 for the SLOTMASK bits);
the library is loaded on first use and a missing library raises. There is no
CPU fallback.

The function names match the C entry points:
    attn_qkv_pack(x, w_qkv, b_q, b_v, out=None)        -> qkv
    attn_qkv_pack_q8_0(x, w_q8_0, b_q, b_v, out=None)  -> qkv
    attn_forward(q, k, v, batch, t_q, t_kv, n_heads, mask=..., out=None) -> out
      (split=False sets ATTN_FLAG_NO_SPLIT)
    attn_forward with sinks=...                          -> attn_forward_sinks
    attn_cross(q, k_enc, v_enc, batch, t_q, t_enc, n_heads, out=None)   -> out
and, on a paged K/V cache (PagedKV),
    attn_paged_append(k_new, v_new, cache, batch, t_new)                -> None
    attn_paged(q, cache, batch, t_q, n_heads, ...)                      -> out [, lse]
    attn_paged_weights(q, cache, lse, batch, t_q, n_heads, weights=...) -> weights
    attn_paged_evict(cache, weights, budget, first, recent, dst=None)   -> kept, weights
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading
from collections import namedtuple
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libattn.so")

ATTN_OK = 0
ATTN_ERR_INVALID = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4

ATTN_FLAG_NO_SPLIT = 1

MASK_FULL = 0
MASK_CHUNK = 1
MASK_SLOTMASK = 2
MASK_BAND = 3

HEAD_DIM = 64
DEFAULT_SCALE = 0.125  # 1/sqrt(64)


class AttnMat(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64)]


class AttnMask(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("chunk_len", ctypes.c_int32),
        ("bits", ctypes.c_void_p),
        ("words_per_row", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("flags", ctypes.c_int32),
        ("q_lens", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p),
    ]


class AttnPlanInfo(ctypes.Structure):
    _fields_ = [
        ("seg_len", ctypes.c_int32),
        ("tiles_per_seg", ctypes.c_int32),
        ("q_tiles", ctypes.c_int32),
        ("kv_splits", ctypes.c_int32),
        ("kv_tiles_per_split", ctypes.c_int32),
        ("proj_tile_n", ctypes.c_int32),
        ("units", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_size_t),
        ("cluster_merge", ctypes.c_int32),
        ("narrow", ctypes.c_int32),
    ]


class AttnPagedKV(ctypes.Structure):
    _fields_ = [
        ("k", AttnMat),
        ("v", AttnMat),
        ("table", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("pages_per_seq", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
    ]


class AttnPagedMask(ctypes.Structure):
    _fields_ = [
        ("window", ctypes.c_int32),
        ("first", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("q_lens", ctypes.c_void_p),
    ]


# (name, restype, argtypes) of every exported entry point.
SIGNATURES = {
    "attn_qkv_pack": (ctypes.c_int, [AttnMat, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_int32, AttnMat, ctypes.c_void_p]),
    "attn_qkv_pack_q8_0": (ctypes.c_int, [AttnMat, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_int32, AttnMat, ctypes.c_void_p]),
    "attn_forward": (ctypes.c_int, [AttnMat, AttnMat, AttnMat, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, AttnMask,
                                    ctypes.c_float, AttnMat, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_void_p]),
    "attn_forward_sinks": (ctypes.c_int, [AttnMat, AttnMat, AttnMat, ctypes.c_int32, ctypes.c_int32,
                                          ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, AttnMask,
                                          ctypes.c_void_p, ctypes.c_float, AttnMat, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p]),
    "attn_cross": (ctypes.c_int, [AttnMat, AttnMat, AttnMat, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                  AttnMat, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "attn_cross_static_scratch": (ctypes.c_int, [AttnMat, AttnMat, AttnMat, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_float, AttnMat, ctypes.c_void_p]),
    "attn_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 6),
    "attn_paged_append": (ctypes.c_int, [AttnMat, AttnMat, AttnPagedKV, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_void_p, ctypes.c_void_p]),
    "attn_paged": (ctypes.c_int, [AttnMat, AttnPagedKV, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, AttnPagedMask,
                                  ctypes.c_void_p, ctypes.c_float, AttnMat, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_size_t, ctypes.c_void_p]),
    "attn_paged_workspace_size": (ctypes.c_size_t, [AttnPagedKV, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                    AttnPagedMask]),
    "attn_paged_weights_workspace_size": (ctypes.c_size_t, [AttnPagedKV, ctypes.c_int32, ctypes.c_int32,
                                                            ctypes.c_int32]),
    "attn_paged_weights": (ctypes.c_int, [AttnMat, AttnPagedKV, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                          AttnPagedMask, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "attn_paged_evict": (ctypes.c_int, [AttnPagedKV, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_void_p, AttnPagedKV, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "attn_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "attn_debug_error_word": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "attn_debug_timeout_probe": (ctypes.c_int, [ctypes.c_int64, ctypes.c_void_p]),
    "attn_debug_plan": (ctypes.c_int, [ctypes.c_int32] * 7 + [ctypes.c_int64, ctypes.c_int32,
                                                              ctypes.POINTER(AttnPlanInfo)]),
}

_lib = None
_lock = threading.Lock()


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load_library(path: str = LIB_PATH):
    """Loads libattn.so (built in-tree by ``python -m speech_encoder_attention_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libattn.so not found at {path}; build it with "
                               "`python -m speech_encoder_attention_b200.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().attn_status_string(status).decode()


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def _stream_ptr(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _mat(t, cols: Optional[int] = None) -> AttnMat:
    """A 2-D CUDA fp16 tensor (or a column view of one) as {ptr, row_stride}."""
    import torch
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor (there is no CPU path)")
    if t.dtype != torch.float16:
        raise ValueError(f"expected float16, got {t.dtype}")
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return AttnMat(t.data_ptr(), stride[0])


def _ptr(t) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor (there is no CPU path)")
    return ctypes.c_void_p(t.data_ptr())


def attn_qkv_pack(x, w_qkv, b_q=None, b_v=None, out=None, stream=None):
    """qkv = x . W^T + [b_q | 0 | b_v].  x [rows, d], W [3d, d] -> [rows, 3d] fp16."""
    import torch
    lib = load_library()
    rows, d = x.shape
    if w_qkv.shape != (3 * d, d) or not w_qkv.is_contiguous() or w_qkv.dtype != torch.float16:
        raise ValueError("w_qkv must be a contiguous [3*d_model, d_model] fp16 tensor")
    for b in (b_q, b_v):
        if b is not None and (b.shape != (d,) or b.dtype != torch.float16 or not b.is_contiguous()):
            raise ValueError("biases must be contiguous [d_model] fp16 tensors")
    if out is None:
        out = torch.empty(rows, 3 * d, dtype=torch.float16, device=x.device)
    st = lib.attn_qkv_pack(_mat(x), _ptr(w_qkv), _ptr(b_q), _ptr(b_v), rows, d, _mat(out),
                           _stream_ptr(stream))
    _check(st, "attn_qkv_pack")
    return out


def attn_qkv_pack_q8_0(x, w_q8_0, b_q=None, b_v=None, out=None, stream=None):
    """qkv = x . W^T + [b_q | 0 | b_v] with Q8_0 weights: w_q8_0 is a contiguous
    uint8 CUDA tensor [3*d, d/32*34] (per block: fp16 scale, 32 int8)."""
    import torch
    lib = load_library()
    rows, d = x.shape
    if w_q8_0.dtype != torch.uint8 or w_q8_0.shape != (3 * d, d // 32 * 34) or not w_q8_0.is_contiguous():
        raise ValueError("w_q8_0 must be a contiguous [3*d_model, d_model/32*34] uint8 tensor")
    for b in (b_q, b_v):
        if b is not None and (b.shape != (d,) or b.dtype != torch.float16 or not b.is_contiguous()):
            raise ValueError("biases must be contiguous [d_model] fp16 tensors")
    if out is None:
        out = torch.empty(rows, 3 * d, dtype=torch.float16, device=x.device)
    st = lib.attn_qkv_pack_q8_0(_mat(x), _ptr(w_q8_0), _ptr(b_q), _ptr(b_v), rows, d, _mat(out),
                                _stream_ptr(stream))
    _check(st, "attn_qkv_pack_q8_0")
    return out


def _lens_ptr(t):
    import torch
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("sequence lengths must be a contiguous [batch] int32 CUDA tensor")
    return _ptr(t).value or 0


def make_mask(kind: int = MASK_FULL, chunk_len: int = 0, bits=None, window: int = 0, causal: bool = False,
              q_lens=None, kv_lens=None) -> AttnMask:
    import torch
    m = AttnMask()
    m.kind = kind
    m.chunk_len = chunk_len
    m.window = window
    m.causal = 1 if causal else 0
    m.flags = 0
    m.q_lens = _lens_ptr(q_lens)
    m.kv_lens = _lens_ptr(kv_lens)
    if kind == MASK_SLOTMASK:
        if bits is None or bits.dtype not in (torch.int32, torch.uint32) or bits.dim() != 2:
            raise ValueError("SLOTMASK needs a [t_q, words_per_row] int32/uint32 CUDA tensor")
        if not bits.is_contiguous():
            raise ValueError("mask bits must be contiguous")
        m.bits = _ptr(bits).value or 0
        m.words_per_row = bits.shape[1]
    else:
        m.bits = 0
        m.words_per_row = 0
    return m


def workspace_size(batch, t_q, t_kv, n_heads, mask_kind=MASK_FULL, head_dim=HEAD_DIM) -> int:
    return int(load_library().attn_workspace_size(batch, t_q, t_kv, n_heads, head_dim, mask_kind))


def _workspace(nbytes: int, device, workspace=None):
    import torch
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def attn_forward(q, k, v, batch, t_q, t_kv, n_heads, mask_kind=MASK_FULL, chunk_len=0, bits=None,
                 scale=DEFAULT_SCALE, out=None, workspace=None, split=True, stream=None, window=0,
                 causal=False, q_lens=None, kv_lens=None, sinks=None):
    """Masked multi-head flash attention. q [batch*t_q, >=H*64] (or a column
    view of the packed qkv buffer), k/v [batch*t_kv, >=H*64]; returns out
    [batch*t_q, H*64] fp16. window / causal / q_lens / kv_lens select the
    range family's band, causal flag and per-sequence lengths ([batch] int32
    CUDA tensors); sinks ([n_heads] fp32 CUDA tensor) calls attn_forward_sinks."""
    import torch
    lib = load_library()
    mask = make_mask(mask_kind, chunk_len, bits, window, causal, q_lens, kv_lens)
    if not split:
        mask.flags = ATTN_FLAG_NO_SPLIT
    if out is None:
        out = torch.empty(batch * t_q, n_heads * HEAD_DIM, dtype=torch.float16, device=q.device)
    need = workspace_size(batch, t_q, t_kv, n_heads, mask_kind) if split else 0
    ws, ws_bytes = _workspace(need, q.device, workspace) if split else (None, 0)
    if sinks is None:
        st = lib.attn_forward(_mat(q), _mat(k), _mat(v), batch, t_q, t_kv, n_heads, HEAD_DIM, mask,
                              float(scale), _mat(out), _ptr(ws), ws_bytes, _stream_ptr(stream))
        _check(st, "attn_forward")
        return out
    if sinks.dtype != torch.float32 or sinks.dim() != 1 or not sinks.is_contiguous():
        raise ValueError("sinks must be a contiguous [n_heads] float32 CUDA tensor")
    st = lib.attn_forward_sinks(_mat(q), _mat(k), _mat(v), batch, t_q, t_kv, n_heads, HEAD_DIM, mask,
                                _ptr(sinks), float(scale), _mat(out), _ptr(ws), ws_bytes, _stream_ptr(stream))
    _check(st, "attn_forward_sinks")
    return out


def attn_cross(q, k_enc, v_enc, batch, t_q, t_enc, n_heads, scale=DEFAULT_SCALE, out=None,
               workspace=None, split=True, stream=None):
    """Decoder queries against every encoder frame (FULL, t_q != t_enc allowed).
    split=False passes no workspace: a split that needs one does not happen, a
    split merged inside a cluster still does (attn_cross takes no flags; use
    attn_forward with split=False for a fixed summation order)."""
    import torch
    lib = load_library()
    if out is None:
        out = torch.empty(batch * t_q, n_heads * HEAD_DIM, dtype=torch.float16, device=q.device)
    need = workspace_size(batch, t_q, t_enc, n_heads, MASK_FULL) if split else 0
    ws, ws_bytes = _workspace(need, q.device, workspace) if split else (None, 0)
    st = lib.attn_cross(_mat(q), _mat(k_enc), _mat(v_enc), batch, t_q, t_enc, n_heads, HEAD_DIM,
                        float(scale), _mat(out), _ptr(ws), ws_bytes, _stream_ptr(stream))
    _check(st, "attn_cross")
    return out


def encoder_layer_attention(x, w_qkv, b_q, b_v, batch, t, n_heads, mask_kind=MASK_FULL,
                            chunk_len=0, qkv=None, out=None, stream=None):
    """The encoder attention pass: packed projection, then attention read in
    place from the packed buffer (q, k, v are column views of it)."""
    d = x.shape[1]
    qkv = attn_qkv_pack(x, w_qkv, b_q, b_v, out=qkv, stream=stream)
    return attn_forward(qkv[:, :d], qkv[:, d:2 * d], qkv[:, 2 * d:], batch, t, t, n_heads,
                        mask_kind=mask_kind, chunk_len=chunk_len, out=out, stream=stream)


# ---------------------------------------------------------------------------
# paged K/V cache
# ---------------------------------------------------------------------------

class PagedKV(namedtuple("PagedKV", "k v table lens page_size n_kv_heads batch slots device c")):
    """A paged K/V cache: pools k and v [num_pages * page_size, n_kv_heads * 64]
    fp16 (column views of one buffer will do), table [batch, pages_per_seq] int32
    (entries outside [0, num_pages) are holes) and lens [batch] int32, the slots
    in use, new tokens included. Slot j of sequence b is row
    table[b, j // page_size] * page_size + j % page_size.

    The tensors are checked here, once, and cannot be exchanged (_replace makes
    another PagedKV, checked anew); what they hold may change at any time (a
    captured graph follows table and lens). batch, slots (per sequence), device
    and c (the C structure) follow from them."""
    __slots__ = ()

    def __new__(cls, k, v, table, lens, page_size: int, n_kv_heads: int):
        import torch
        if page_size not in (16, 32, 64, 128, 256):
            raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, got {page_size}")
        if n_kv_heads < 1:
            raise ValueError("n_kv_heads must be positive")
        cols = n_kv_heads * HEAD_DIM
        (k_ptr, rows, k_stride), (v_ptr, v_rows, v_stride) = _half_rows(k, "k", cols), _half_rows(v, "v", cols)
        dev = k.device
        if v.device != dev or v_rows != rows:
            raise ValueError("the K and V pools must lie on one device and have as many rows")
        if rows == 0 or rows % page_size:
            raise ValueError(f"the pools must hold whole pages of {page_size} rows")
        shape = table.shape
        if len(shape) != 2:
            raise ValueError("table must be a [batch, pages_per_seq] int32 tensor")
        batch, per_seq = shape
        table_ptr = _dev_tensor(table, "table", torch.int32, shape, dev)
        lens_ptr = _dev_tensor(lens, "lens", torch.int32, (batch,), dev)
        c = AttnPagedKV.from_buffer_copy(_PAGED_KV.pack(k_ptr, k_stride, v_ptr, v_stride, table_ptr, lens_ptr,
                                                        rows // page_size, page_size, per_seq, n_kv_heads))
        return tuple.__new__(cls, (k, v, table, lens, page_size, n_kv_heads, batch, per_seq * page_size, dev, c))

    # Every way to another PagedKV goes through the checks: c holds addresses.

    def __getnewargs__(self):
        return tuple(self[:6])

    def _replace(self, **changes):
        """This cache with some of k, v, table, lens, page_size and n_kv_heads exchanged, checked as a new one."""
        given = dict(zip(self._fields, self[:6]))
        other = [name for name in changes if name not in given]
        if other:
            raise ValueError(f"a PagedKV is made of {', '.join(given)}, not of {', '.join(other)}")
        return type(self)(**{**given, **changes})

    __replace__ = _replace

    @classmethod
    def _make(cls, iterable):
        raise TypeError("a PagedKV is made from its tensors: PagedKV(k, v, table, lens, page_size, n_kv_heads)")


_INT_MAX = 2 ** 31 - 1
_PAGED_KV = struct.Struct("@QqQqQQiiii")  # the fields of AttnPagedKV, in order


def _half_rows(t, what: str, cols: int):
    """(pointer, rows, row stride) of a 2-D CUDA fp16 tensor of at least cols columns, or a column view of one."""
    import torch
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (there is no CPU path)")
    if t.dtype is not torch.float16:
        raise ValueError(f"{what} must be float16, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] < cols or stride[1] != 1:
        raise ValueError(f"{what} must be 2-D with unit column stride and at least {cols} columns, got {list(shape)}")
    return t.data_ptr(), shape[0], stride[0]


def _dev_tensor(t, what: str, dtype, shape, device) -> int:
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the cache on {device}")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {list(shape)} {dtype} tensor, got {list(t.shape)} {t.dtype}")
    return t.data_ptr()


def _rows(t, what: str, rows: int, cols: int, device) -> AttnMat:
    ptr, have, stride = _half_rows(t, what, cols)
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the cache on {device}")
    if have != rows:
        raise ValueError(f"{what} must have {rows} rows, got {have}")
    return AttnMat(ptr, stride)


def _paged_mask(window: int, first: int, causal, q_lens, batch: int, device) -> AttnPagedMask:
    if not (0 <= window <= _INT_MAX and 0 <= first <= _INT_MAX):
        raise ValueError(f"window and first must be 32-bit and not negative, got {window} and {first}")
    return AttnPagedMask(window, first, 1 if causal else 0, _q_lens_ptr(q_lens, batch, device))


def _sizes_fit(t_q: int, n_heads: int) -> None:
    if not (0 < t_q <= _INT_MAX and 0 < n_heads <= _INT_MAX):
        raise ValueError(f"t_q and n_heads must be positive and 32-bit, got {t_q} and {n_heads}")


def _batch_of(cache: PagedKV, batch: int) -> AttnPagedKV:
    if batch != cache.batch:
        raise ValueError(f"the cache holds {cache.batch} sequences, not {batch}")
    return cache.c


def _q_lens_ptr(q_lens, batch, device) -> int:
    import torch
    return 0 if q_lens is None else _dev_tensor(q_lens, "q_lens", torch.int32, (batch,), device)


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device and the call's stream as the current ones, so that
    what is allocated and launched belongs to them."""
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {device}")
        with torch.cuda.stream(stream):
            yield


def _elsewhere(torch, device, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    return stream is not None or torch._C._cuda_getDevice() != device.index


def attn_paged_append(k_new, v_new, cache: PagedKV, batch, t_new, q_lens=None, stream=None) -> None:
    """Writes a chunk's K and V rows ([batch*t_new, n_kv_heads*64] fp16, or column
    views) into the slots at the end of each sequence; cache.lens already counts
    them, q_lens ([batch] int32) says how many of the t_new rows are valid."""
    import torch
    dev, cols = cache.device, cache.n_kv_heads * HEAD_DIM
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return attn_paged_append(k_new, v_new, cache, batch, t_new, q_lens)
    kv = _batch_of(cache, batch)
    kn, vn = _rows(k_new, "k_new", batch * t_new, cols, dev), _rows(v_new, "v_new", batch * t_new, cols, dev)
    lens = _q_lens_ptr(q_lens, batch, dev)
    st = load_library().attn_paged_append(kn, vn, kv, batch, t_new, lens, torch._C._cuda_getCurrentRawStream(dev.index))
    _check(st, "attn_paged_append")


def paged_workspace_size(cache: PagedKV, batch, t_q, n_heads, window=0, first=0, causal=True) -> int:
    """Bytes of workspace attn_paged needs for these sizes on the current device."""
    _sizes_fit(t_q, n_heads)
    mask = _paged_mask(window, first, causal, None, batch, cache.device)
    return int(load_library().attn_paged_workspace_size(_batch_of(cache, batch), batch, t_q, n_heads, mask))


def paged_weights_workspace_size(cache: PagedKV, batch, t_q, n_heads) -> int:
    """Bytes of workspace attn_paged_weights needs for these sizes on the current device."""
    _sizes_fit(t_q, n_heads)
    return int(load_library().attn_paged_weights_workspace_size(_batch_of(cache, batch), batch, t_q, n_heads))


def _given_workspace(workspace, device):
    """A caller's workspace as (pointer, bytes)."""
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the cache on {device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def attn_paged(q, cache: PagedKV, batch, t_q, n_heads, window=0, first=0, causal=True, q_lens=None, sinks=None,
               scale=DEFAULT_SCALE, out=None, return_lse=False, lse=None, workspace=None, stream=None):
    """Attention of a chunk of new tokens (t_q = 1: a decode step) over a paged
    cache; q [batch*t_q, >= n_heads*64] fp16. window and first limit what a row
    sees to the last `window` slots and the `first` first ones (window=0: all).
    Returns out, or (out, lse) with return_lse or lse given; lse is
    [batch*t_q, n_heads] fp32, the log of each row's softmax denominator.
    Without workspace one is allocated for the call, if it needs any."""
    import torch
    dev, rows, cols = cache.device, batch * t_q, n_heads * HEAD_DIM
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return attn_paged(q, cache, batch, t_q, n_heads, window, first, causal, q_lens, sinks, scale, out,
                              return_lse, lse, workspace)
    lib = load_library()
    kv = _batch_of(cache, batch)
    qm = _rows(q, "q", rows, cols, dev)
    mask = _paged_mask(window, first, causal, q_lens, batch, dev)
    sinks_ptr = 0 if sinks is None else _dev_tensor(sinks, "sinks", torch.float32, (n_heads,), dev)
    if out is None:
        out = torch.empty_like(q) if q.shape[1] == cols and q.is_contiguous() else q.new_empty((rows, cols))
        om = AttnMat(out.data_ptr(), cols)
    else:
        om = _rows(out, "out", rows, cols, dev)
    if lse is not None:
        lse_ptr = _dev_tensor(lse, "lse", torch.float32, (rows, n_heads), dev)
    elif return_lse:
        lse = q.new_empty((rows, n_heads), dtype=torch.float32)
        lse_ptr = lse.data_ptr()
    else:
        lse_ptr = 0
    if workspace is not None:
        ws_ptr, ws_bytes = _given_workspace(workspace, dev)
    else:
        ws_ptr, ws_bytes = 0, lib.attn_paged_workspace_size(kv, batch, t_q, n_heads, mask)
        if ws_bytes:
            workspace = q.new_empty(ws_bytes, dtype=torch.uint8)
            ws_ptr = workspace.data_ptr()
    st = lib.attn_paged(qm, kv, batch, t_q, n_heads, mask, sinks_ptr, scale, om, lse_ptr, ws_ptr, ws_bytes,
                        torch._C._cuda_getCurrentRawStream(dev.index))
    _check(st, "attn_paged")
    return out if lse is None else (out, lse)


def attn_paged_weights(q, cache: PagedKV, lse, batch, t_q, n_heads, window=0, first=0, causal=True, q_lens=None,
                       scale=DEFAULT_SCALE, weights=None, out=None, workspace=None, stream=None):
    """What attn_paged's rows put on each slot, summed over rows and heads, added
    to weights ([batch, cache.slots] fp32; None: zeros). lse is attn_paged's.
    Returns out, a new tensor unless given; out=weights adds in place. Without
    workspace one is allocated for the call, if it needs any."""
    import torch
    dev, rows = cache.device, batch * t_q
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return attn_paged_weights(q, cache, lse, batch, t_q, n_heads, window, first, causal, q_lens, scale, weights,
                                      out, workspace)
    lib = load_library()
    kv = _batch_of(cache, batch)
    qm = _rows(q, "q", rows, n_heads * HEAD_DIM, dev)
    mask = _paged_mask(window, first, causal, q_lens, batch, dev)
    lse_ptr = _dev_tensor(lse, "lse", torch.float32, (rows, n_heads), dev)
    shape = (batch, cache.slots)
    w_in = 0 if weights is None else _dev_tensor(weights, "weights", torch.float32, shape, dev)
    if out is None:
        out = lse.new_empty(shape)
    w_out = _dev_tensor(out, "out", torch.float32, shape, dev)
    if workspace is not None:
        ws_ptr, ws_bytes = _given_workspace(workspace, dev)
    else:
        ws_ptr, ws_bytes = 0, lib.attn_paged_weights_workspace_size(kv, batch, t_q, n_heads)
        if ws_bytes:
            workspace = lse.new_empty(ws_bytes, dtype=torch.uint8)
            ws_ptr = workspace.data_ptr()
    st = lib.attn_paged_weights(qm, kv, batch, t_q, n_heads, mask, lse_ptr, scale, w_in, w_out, ws_ptr, ws_bytes,
                                torch._C._cuda_getCurrentRawStream(dev.index))
    _check(st, "attn_paged_weights")
    return out


def attn_paged_evict(cache: PagedKV, weights, budget, first=0, recent=0, dst: Optional[PagedKV] = None, kept=None,
                     weights_out=None, stream=None):
    """Shrinks each sequence to its `first` first, `recent` last and heaviest
    slots, `budget` in all, in order, at the front of dst (None: in place, in
    cache's own pages; cache.lens is updated). dst's table must have a page for
    each of the first `budget` slots: what would go to a hole is lost. Returns (kept, weights):
    kept [batch, budget] int32 holds the old slot of each new one (-1 behind the
    last), weights [batch, dst slots] the moved weights (0 behind the last).
    dst.lens is written. Without weights_out a new tensor is returned;
    weights_out=weights works in place when dst has as many slots."""
    import torch
    batch, dev = cache.batch, cache.device
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return attn_paged_evict(cache, weights, budget, first, recent, dst, kept, weights_out)
    if dst is None:
        dst = cache
    elif dst.device != dev:
        raise ValueError(f"dst is on {dst.device}, the cache on {dev}")
    if not (0 <= budget <= _INT_MAX and 0 <= first <= _INT_MAX and 0 <= recent <= _INT_MAX):
        raise ValueError(f"budget, first and recent must be 32-bit and not negative, got {budget}, {first} and {recent}")
    to = _batch_of(dst, batch)
    w_in = _dev_tensor(weights, "weights", torch.float32, (batch, cache.slots), dev)
    if kept is None:
        kept = weights.new_empty((batch, budget), dtype=torch.int32)
    if weights_out is None:
        weights_out = weights.new_empty((batch, dst.slots))
    w_out = _dev_tensor(weights_out, "weights_out", torch.float32, (batch, dst.slots), dev)
    st = load_library().attn_paged_evict(cache.c, batch, budget, first, recent, w_in, to, w_out,
                                         _dev_tensor(kept, "kept", torch.int32, (batch, budget), dev),
                                         torch._C._cuda_getCurrentRawStream(dev.index))
    _check(st, "attn_paged_evict")
    return kept, weights_out


def debug_error_word(stream=None):
    """Synchronises the stream; returns (status, raw word) and clears the word."""
    w = ctypes.c_uint32(0)
    st = load_library().attn_debug_error_word(_stream_ptr(stream), ctypes.byref(w))
    return st, w.value


def debug_timeout_probe(limit_ns: int, stream=None) -> int:
    return load_library().attn_debug_timeout_probe(int(limit_ns), _stream_ptr(stream))


def debug_plan(batch, t_q, t_kv, n_heads, mask_kind=MASK_FULL, chunk_len=0, num_sms=148, proj_rows=0,
               d_model=0) -> dict:
    """The launch plan the library would choose on a GPU with num_sms SMs (host arithmetic only)."""
    info = AttnPlanInfo()
    st = load_library().attn_debug_plan(batch, t_q, t_kv, n_heads, mask_kind, chunk_len, num_sms, proj_rows,
                                        d_model, ctypes.byref(info))
    _check(st, "attn_debug_plan")
    return {name: getattr(info, name) for name, _ in AttnPlanInfo._fields_}
