"""Paged KV cache: append with rotary positions, attention of new tokens and
decode attention over it (the paged-cache section of include/up.h).

    cache = PagedKV(k_pages, v_pages, block_table, kv_lens, pos_pages)
    q = append_kv(q, k, v, pos, cu_seqlens, cache, inv_freq)
    out, lse = attend_paged(q, cu_seqlens, cache)       # a chunk of new tokens
    out, lse = decode_attend(q, cache)                  # one new token per sequence
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1}
ROPE_INTERLEAVED = 0x1


class _CKv(ctypes.Structure):
    """up_paged_kv of include/up.h."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("pos_pages", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("kv_lens", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("num_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hk", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _CLogits(ctypes.Structure):
    """up_logits of include/up.h."""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("slopes", ctypes.c_void_p), ("q_pos", ctypes.c_void_p)]


_lib = None


def _L():
    """The loaded library (looked up once: a decode step's calls are short)."""
    global _lib
    if _lib is None:
        from . import lib
        _lib = lib()
    return _lib


def _error(where, status):
    from . import UpError
    return UpError(where, status)


def _refuse(t, name, dtype, device, shape=None):
    """Raises what is wrong with tensor t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _need(t, name, dtype, device, shape=None):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous()
            and (device is None or t.device == device) and (shape is None or t.shape == shape)):
        _refuse(t, name, dtype, device, shape)


class PagedKV:
    """A paged KV-head-major cache: k_pages and v_pages [num_pages, Hk, page_size, d]
    (bf16 or fp16), block_table int32 [num_seqs, max_pages], kv_lens int32
    [num_seqs] (cached tokens, those of the current call included) and, where
    positions matter, pos_pages int32 [num_pages, page_size].  Holds the tensors;
    their contents may change between calls (an engine adds to kv_lens and to
    block_table in place), the attributes and the tensors' storage may not: other
    tensors are another PagedKV."""

    __slots__ = ("k_pages", "v_pages", "block_table", "kv_lens", "pos_pages", "num_seqs", "Hk", "d",
                 "page_size", "dtype", "device", "struct", "ref")

    def __init__(self, k_pages, v_pages, block_table, kv_lens, pos_pages=None):
        if not isinstance(k_pages, torch.Tensor):
            raise TypeError("k_pages must be a torch.Tensor")
        dt, dev = k_pages.dtype, k_pages.device
        if dt not in DTYPES:
            raise TypeError(f"k_pages must be bfloat16 or float16, got {dt}")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [num_pages, Hk, page_size, d]")
        _need(k_pages, "k_pages", dt, None)
        _need(v_pages, "v_pages", dt, dev, k_pages.shape)
        _need(block_table, "block_table", torch.int32, dev)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [num_seqs, max_pages]")
        n, hk, ps, d = k_pages.shape
        b, mp = block_table.shape
        _need(kv_lens, "kv_lens", torch.int32, dev, (b,))
        if pos_pages is not None:
            _need(pos_pages, "pos_pages", torch.int32, dev, (n, ps))
        c = _CKv(k_pages.data_ptr(), v_pages.data_ptr(),
                 None if pos_pages is None else pos_pages.data_ptr(), block_table.data_ptr(),
                 kv_lens.data_ptr(), n, b, mp, ps, hk, d, DTYPES[dt])
        for put, x in zip(_PUT, (k_pages, v_pages, block_table, kv_lens, pos_pages, b, hk, d, ps, dt,
                                 dev, c, ctypes.byref(c))):
            put(self, x)

    def _fixed(self, name, value=None):
        raise AttributeError(f"{name}: a PagedKV's attributes are fixed")

    __setattr__ = __delattr__ = _fixed

    def __reduce__(self):  # copies go through the checks and get a struct of their own
        return type(self), (self.k_pages, self.v_pages, self.block_table, self.kv_lens, self.pos_pages)

    def __repr__(self):
        return (f"PagedKV({self.k_pages.shape[0]} pages of {self.page_size} slots, {self.Hk} heads of "
                f"{self.d}, {self.dtype}, {self.num_seqs} sequences)")


_PUT = tuple(PagedKV.__dict__[name].__set__ for name in PagedKV.__slots__)


def _on(stream):
    """Allocations of a call on `stream` belong to that stream, so a workspace
    freed on return is not handed to another stream's work while it is in use."""
    return _HERE if stream is None else torch.cuda.stream(stream)


_HERE = contextlib.nullcontext()


def _raw(stream, device):
    if torch._C._cuda_getDevice() != device.index:
        raise ValueError(f"the current device is not the tensors' {device}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream


def _rows(t, name, cache, heads=None):
    """Token stride of a [tokens, heads, d] tensor whose heads are adjacent (a view
    of a fused projection is fine)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype}, got {t.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, expected {cache.device}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.d or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {cache.d}], got {tuple(shape)}")
    st, sh, sd = t.stride()
    if sd != 1 or (sh != cache.d and shape[1] > 1):
        raise ValueError(f"{name}'s heads must be adjacent")
    return shape[1] * cache.d if shape[0] < 2 else st


def append_kv(q, k, v, pos, cu_seqlens, cache, inv_freq, axes=None, interleaved=False, q_out=None,
              stream=None):
    """Rotates q and k by their positions, writes k, v and the positions to the
    cache and returns the rotated q (see up_append_kv).

    q [T, Hq, d] or None, k and v [T, Hk, d] (heads adjacent, any token stride that
    is a multiple of 8); pos int32 [T] or [num_axes, T]; cu_seqlens int32
    [num_seqs + 1] over the new tokens; cache a PagedKV whose kv_lens already count
    them; inv_freq fp32 [rot_dim / 2] (None: no rotation); axes int32 [rot_dim / 2],
    the row of pos that turns each frequency; interleaved: pairs (2i, 2i+1) instead
    of (i, i + rot_dim/2); q_out [T, Hq, d] (q itself is allowed)."""
    dev = cache.device
    ks, vs = _rows(k, "k", cache, cache.Hk), _rows(v, "v", cache, cache.Hk)
    T, Hq, qs = k.shape[0], 0, 0
    if v.shape[0] != T:
        raise ValueError("k and v must have the same tokens")
    if q is not None:
        qs = _rows(q, "q", cache)
        Hq = q.shape[1]
        if q.shape[0] != T:
            raise ValueError("q and k must have the same tokens")
    _need(pos, "pos", torch.int32, dev)
    A = 1 if pos.dim() == 1 else pos.shape[0]
    if pos.dim() not in (1, 2) or pos.shape[-1] != T or A < 1:
        raise ValueError("pos must be [tokens] or [num_axes, tokens]")
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.num_seqs + 1,))
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, dev)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot_dim / 2]")
        rot = 2 * inv_freq.numel()
    if axes is not None:
        _need(axes, "axes", torch.int32, dev, (rot // 2,))
    with _on(stream):
        if q is not None:
            if q_out is None:
                q_out = torch.empty((T, Hq, cache.d), dtype=cache.dtype, device=dev)
            elif q_out is not q:
                _need(q_out, "q_out", cache.dtype, dev, q.shape)
        elif q_out is not None:
            raise ValueError("q_out without q")
        st = _L().up_append_kv(
            None if q is None else q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
            pos.data_ptr(), A, None if axes is None else axes.data_ptr(),
            None if inv_freq is None else inv_freq.data_ptr(), rot,
            ROPE_INTERLEAVED if interleaved else 0, cu_seqlens.data_ptr(), T, Hq, cache.ref,
            None if q is None else q_out.data_ptr(), _raw(stream, dev))
    if st:
        raise _error("up_append_kv", st)
    return q_out


@functools.lru_cache(maxsize=64)
def _plain_logits(scale, softcap):
    lg = _CLogits(scale, softcap, None, None)  # read by the library during a call, never written
    return ctypes.byref(lg)


def _logits(cache, T, Hq, scale, softcap, slopes, q_pos):
    # plain numbers: a tensor would be remembered by its identity, with its first value
    if type(scale) is not float:
        scale = ctypes.c_float(scale).value
    if type(softcap) is not float:
        softcap = ctypes.c_float(softcap).value
    if slopes is None:
        return _plain_logits(scale, softcap)
    _need(slopes, "slopes", torch.float32, cache.device, (Hq,))
    if q_pos is None or cache.pos_pages is None:
        raise ValueError("slopes need q_pos and a cache with pos_pages")
    _need(q_pos, "q_pos", torch.int32, cache.device, (T,))
    return ctypes.byref(_CLogits(scale, softcap, slopes.data_ptr(), q_pos.data_ptr()))


def _given(out, lse, workspace, cache, shape):
    """Checks the buffers that the caller brought."""
    if out is not None:
        _need(out, "out", cache.dtype, cache.device, shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, cache.device, shape[:2])
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if workspace.device != cache.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {cache.device}")


@functools.lru_cache(maxsize=256)
def attend_paged_workspace(total_tokens, num_seqs, Hq, Hk, d) -> int:
    """Bytes of attend_paged's workspace (0: sizes it does not take)."""
    return int(_L().up_attend_paged_workspace(total_tokens, num_seqs, Hq, Hk, d))


@functools.lru_cache(maxsize=256)
def decode_attend_workspace(num_seqs, Hq, Hk, d) -> int:
    """Bytes of decode_attend's workspace (0: sizes it does not take)."""
    return int(_L().up_decode_attend_workspace(num_seqs, Hq, Hk, d))


def attend_paged(q, cu_seqlens, cache, scale=None, softcap=0.0, slopes=None, q_pos=None,
                 visible=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens q [T, Hq, d] (packed by cu_seqlens int32
    [num_seqs + 1]) over the cache, which holds their own keys too; returns (out
    [T, Hq, d], lse fp32 [T, Hq]).  See up_attend_paged.

    scale (default d ** -0.5), softcap (0: none); slopes fp32 [Hq] with q_pos int32
    [T]: a bias of -slope * |q_pos - key position|; visible int32 [T, 2]: the slots
    [first, end) each query sees (default: causal)."""
    dev = cache.device
    if _rows(q, "q", cache) != q.shape[1] * cache.d:
        raise ValueError("q must be contiguous")
    T, Hq, d = q.shape
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, (cache.num_seqs + 1,))
    lg = _logits(cache, T, Hq, d ** -0.5 if scale is None else scale, softcap, slopes, q_pos)
    if visible is not None:
        _need(visible, "visible", torch.int32, dev, (T, 2))
    if out is not None or lse is not None or workspace is not None:
        _given(out, lse, workspace, cache, q.shape)
    with _on(stream):
        if out is None:
            out = torch.empty((T, Hq, d), dtype=cache.dtype, device=dev)
        if lse is None:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        if workspace is None:
            size = attend_paged_workspace(T, cache.num_seqs, Hq, cache.Hk, d)
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        else:
            size = workspace.numel() * workspace.element_size()
        st = _L().up_attend_paged(q.data_ptr(), cu_seqlens.data_ptr(), T, Hq, cache.ref, lg,
                             None if visible is None else visible.data_ptr(),
                             out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), size,
                             _raw(stream, dev))
    if st:
        raise _error("up_attend_paged", st)
    return out, lse


def decode_attend(q, cache, scale=None, softcap=0.0, slopes=None, q_pos=None, kv_start=None,
                  out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [num_seqs, Hq, d], over the cache;
    returns (out, lse fp32 [num_seqs, Hq]).  See up_decode_attend.  kv_start int32
    [num_seqs]: the first visible slot of each sequence; the other arguments are
    attend_paged's."""
    dev = cache.device
    if _rows(q, "q", cache) != q.shape[1] * cache.d:
        raise ValueError("q must be contiguous")
    B, Hq, d = q.shape
    if B != cache.num_seqs:
        raise ValueError(f"q must hold one token for each of the {cache.num_seqs} sequences")
    lg = _logits(cache, B, Hq, d ** -0.5 if scale is None else scale, softcap, slopes, q_pos)
    if kv_start is not None:
        _need(kv_start, "kv_start", torch.int32, dev, (B,))
    if out is not None or lse is not None or workspace is not None:
        _given(out, lse, workspace, cache, q.shape)
    with _on(stream):
        if out is None:
            out = torch.empty((B, Hq, d), dtype=cache.dtype, device=dev)
        if lse is None:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        if workspace is None:
            size = decode_attend_workspace(B, Hq, cache.Hk, d)
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        else:
            size = workspace.numel() * workspace.element_size()
        st = _L().up_decode_attend(q.data_ptr(), Hq, cache.ref, lg,
                             None if kv_start is None else kv_start.data_ptr(),
                             out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), size,
                             _raw(stream, dev))
    if st:
        raise _error("up_decode_attend", st)
    return out, lse
