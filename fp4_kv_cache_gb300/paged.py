"""Binding of the paged-cache calls of libcsa2.so (include/csa2_paged.h).

As in ``csa2``: the helpers check what they are given, allocate outputs with torch and call the C
entry points, and everything is computed by the library's kernels.  Work goes to the current
CUDA stream (or the one given: what a call allocates then belongs to that stream), on the current
device, which has to be the tensors'.

A decode step's calls take a few microseconds each on the GPU, so the way there is kept short:
argument structures are packed with ``struct`` (the ctypes classes below name their fields and
are checked against the C compiler's sizes in the tests).
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import csa2
from .csa2 import Csa2Error

MXFP4, NVFP4_E4M3_16, MXFP8, BF16 = 0, 1, 2, 3
DEV_NO_PAGES, DEV_TABLE_FULL, DEV_ROWS = 0x100, 0x200, 0x400
MAX_BATCH = 16384

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_i32, _bf16, _f32, _u8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
# (a torch without CUDA has neither; nothing there gets as far as a stream)
_raw_stream, _device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


class CacheArgs(ctypes.Structure):
    """csa2p_cache"""
    _fields_ = [("fmt", _I32), ("d", _I32), ("page", _I32), ("n_pages", _I64), ("codes", _P), ("scales", _P),
                ("code_stride", _I64), ("scale_stride", _I64)]


class PlanArgs(ctypes.Structure):
    """csa2p_plan_args"""
    _fields_ = [("batch", _I32), ("page", _I32), ("width", _I32), ("free_cap", _I32), ("n_rows", _I32), ("lens", _P),
                ("delta", _P), ("lens_out", _P), ("block_table", _P), ("free_pages", _P), ("n_free", _P),
                ("n_free_out", _P), ("cu", _P), ("slot", _P), ("row_req", _P), ("row_pos", _P)]


class RopeAxes(ctypes.Structure):
    """csa2p_rope_axes"""
    _fields_ = [("rope_dim", _I32), ("n_axes", _I32), ("section", _I32 * 3), ("pos", _P), ("cos_sin", _P),
                ("n_pos", _I64)]


class AttnArgs(ctypes.Structure):
    """csa2p_attn_args"""
    _fields_ = [("cache", CacheArgs), ("batch", _I32), ("n_tokens", _I32), ("n_heads", _I32), ("d_v", _I32),
                ("width", _I32), ("window", _I32), ("ratio_m", _I32), ("sm_scale", _F), ("q", _P), ("block_table", _P),
                ("lens", _P), ("cu", _P), ("pos0", _P), ("kv_start", _P)]


_CACHE = "iii4xqPPqq"                                  # csa2p_cache
_PLAN = struct.Struct("@5i4x11P")                      # csa2p_plan_args
_ROPE = struct.Struct("@5i4xPPq")                      # csa2p_rope_axes
_ATTN = struct.Struct("@" + _CACHE + "7if6P")          # csa2p_attn_args
_CACHE = struct.Struct("@" + _CACHE)

_FORMATS = {16: MXFP4, 8: NVFP4_E4M3_16, 32: MXFP8}      # by codes a scale

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = csa2.load()
        S, sz, A = ctypes.c_int, ctypes.c_size_t, _P       # A: an argument structure
        for name, res, args in (
                ("csa2p_page_plan", S, [A, _P, _P]),
                ("csa2p_rope", S, [_P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _I32, A, _P, _P]),
                ("csa2p_write", S, [A, _P, _I64, _I32, _P, A, _P, _P]),
                ("csa2p_read", S, [A, _P, _I32, _P, _I64, _P, _P]),
                ("csa2p_attn_workspace_size", sz, [A]),
                ("csa2p_attn", S, [A, _P, _P, _P, sz, _P, _P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _ready = lib
    return _ready


def _stream_of(dev: int, stream):
    """Raw stream of a call on device `dev`: the one given, else the current one.  The library works
    on the current device, so that has to be the tensors'."""
    if dev != _device():
        raise ValueError(f"the tensors are on cuda:{dev}: make it the current device (torch.cuda.device)")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _bad(t, name: str, dtype, n: Optional[int], dev: int):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on {'the GPU' if dev < 0 else f'cuda:{dev}'}, not {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must hold {n} values, not {t.numel()} ({tuple(t.shape)})")


def _need(t, name: str, dtype, n: Optional[int], dev: int) -> int:
    """Address of a contiguous tensor of this type, size and device."""
    if t.dtype is not dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous() or (n is not None and t.numel() != n):
        _bad(t, name, dtype, n, dev)
    return t.data_ptr()


def _maybe(t, name: str, dtype, n: Optional[int], dev: int) -> int:
    return 0 if t is None else _need(t, name, dtype, n, dev)


def _empty(shape, dtype, device, stream):
    """A new tensor of a call: of the given stream's memory, so that no block is written there that
    another stream has not done with."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status(d_status, dev: int):
    return None if d_status is None else _need(d_status, "d_status", _i32, None, dev)


class PagedCache:
    """One layer's pages: codes [n_pages, page, row bytes] uint8 and scales [n_pages, page, scales a
    row] uint8 (told apart by their widths: MXFP4, E2M1 + E4M3/16, or MXFP8), or bf16 values
    [n_pages, page, d] without scales.  Rows are contiguous within a page; pages may lie apart
    (a view of a larger buffer)."""

    def __init__(self, codes: torch.Tensor, scales: Optional[torch.Tensor] = None):
        shape = codes.shape
        if len(shape) != 3:
            raise ValueError("codes and scales are [n_pages, page, bytes of a row]")
        n, page, w = shape
        index = codes.get_device()                    # -1: not on a GPU
        if scales is None:
            if codes.dtype is not _bf16:
                raise ValueError("a cache without scales holds bf16 values")
            fmt, d, at_scales, scale_pages = BF16, w, 0, 0
        else:
            more = scales.shape
            if len(more) != 3 or more[0] != n or more[1] != page:
                raise ValueError("codes and scales are [n_pages, page, bytes of a row]")
            if codes.dtype is not _u8 or scales.dtype is not _u8 or scales.get_device() != index or (index < 0 and scales.device != codes.device):
                raise ValueError("codes and scales are uint8 tensors on one device")
            fmt = _FORMATS.get(w / more[2] if more[2] else 0)
            if fmt is None:
                raise ValueError("the widths of codes and scales fit no row format")
            d = w if fmt == MXFP8 else 2 * w
            at_scales, scale_pages = scales.data_ptr(), self._pages(scales, n, page, more[2])
        code_pages = self._pages(codes, n, page, w)
        self.codes, self.scales, self.fmt, self.d, self.page, self.n_pages = codes, scales, fmt, d, page, n
        self.device = codes.device
        self.index = index
        self.fields = (fmt, d, page, n, codes.data_ptr(), at_scales, 2 * code_pages if fmt == BF16 else code_pages, scale_pages)
        self.packed = _CACHE.pack(*self.fields)

    @staticmethod
    def _pages(t, n: int, page: int, w: int) -> int:
        """Elements between pages; 0 where there is one."""
        pages, rows, elements = t.stride()
        if elements != 1 or rows != w:
            raise ValueError("rows must be contiguous within a page")
        if n < 2:
            return 0
        # an expanded tensor's stride of 0 would be taken for dense pages, past its storage
        if pages < page * w:
            raise ValueError("pages must not overlap")
        return pages

    def _on_gpu(self) -> int:
        if self.index < 0:
            raise ValueError("libcsa2 takes device tensors (got a CPU cache)")
        return self.index

    @staticmethod
    def new(n_pages: int, page: int, d: int, fmt: int = MXFP4, device="cuda") -> "PagedCache":
        """An empty cache (every byte 0)."""
        if fmt == BF16:
            return PagedCache(torch.zeros((n_pages, page, d), dtype=torch.bfloat16, device=device))
        codes = torch.zeros((n_pages, page, d if fmt == MXFP8 else d // 2), dtype=torch.uint8, device=device)
        g = 16 if fmt == NVFP4_E4M3_16 else 32
        return PagedCache(codes, torch.zeros((n_pages, page, d // g), dtype=torch.uint8, device=device))


@dataclass
class PagePlan:
    """What csa2p_page_plan says of one step (int32 tensors)."""
    lens: torch.Tensor        # [batch] rows held after the step
    cu: torch.Tensor          # [batch + 1] first new row of each request
    slot: torch.Tensor        # [n_rows] cache slot of each new row, -1 past the last
    row_req: torch.Tensor     # [n_rows] its request
    row_pos: torch.Tensor     # [n_rows] its position in the request
    n_free: torch.Tensor      # [1] free pages left


def page_plan(lens, delta, block_table, free_pages, n_free, page: int, n_rows: int, in_place: bool = False,
              plan: Optional[PagePlan] = None, d_status=None, stream=None) -> PagePlan:
    """One step of the requests' bookkeeping: block_table [batch, width] and free_pages are updated,
    the rest is returned (into `plan`'s tensors when given).  in_place: lens and n_free are
    overwritten with the new lengths and the new count, as a captured graph needs it (a plan given
    with it holds these two tensors).  See csa2p_page_plan."""
    dev, B = lens.get_device(), lens.shape[0]
    width = block_table.shape[1]
    if plan is None:
        # one allocation: lens | n_free | cu | slot | row_req | row_pos
        buf = _empty(2 * B + 2 + 3 * n_rows, _i32, lens.device, stream)
        parts = torch.split_with_sizes(buf, (B, 1, B + 1, n_rows, n_rows, n_rows))
        base = buf.data_ptr()
        at_cu, at_slot = base + 4 * B + 4, base + 8 * B + 8
        if in_place:
            plan = PagePlan(lens, parts[2], parts[3], parts[4], parts[5], n_free)
            at_len, at_n = lens.data_ptr(), n_free.data_ptr()
        else:
            plan = PagePlan(parts[0], parts[2], parts[3], parts[4], parts[5], parts[1])
            at_len, at_n = base, base + 4 * B
        at_req, at_pos = at_slot + 4 * n_rows, at_slot + 8 * n_rows
    else:
        at_len, at_n = _need(plan.lens, "plan.lens", _i32, B, dev), _need(plan.n_free, "plan.n_free", _i32, 1, dev)
        at_cu, at_slot = _need(plan.cu, "plan.cu", _i32, B + 1, dev), _need(plan.slot, "plan.slot", _i32, n_rows, dev)
        at_req, at_pos = _need(plan.row_req, "plan.row_req", _i32, n_rows, dev), _need(plan.row_pos, "plan.row_pos", _i32, n_rows, dev)
        if in_place and (at_len != lens.data_ptr() or at_n != n_free.data_ptr()):
            raise ValueError("in_place: plan.lens and plan.n_free must be lens and n_free")
    a = _PLAN.pack(B, page, width, free_pages.shape[0], n_rows, _need(lens, "lens", _i32, B, dev),
                   _need(delta, "delta", _i32, B, dev), at_len, _need(block_table, "block_table", _i32, B * width, dev),
                   _need(free_pages, "free_pages", _i32, None, dev), _need(n_free, "n_free", _i32, 1, dev), at_n, at_cu, at_slot,
                   at_req, at_pos)
    st = (_ready or _lib()).csa2p_page_plan(a, _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2p_page_plan", st)
    return plan


def _axes(pos, cos_sin, sections, rows: int, dev: int):
    """csa2p_rope_axes of pos int32 [rows] or [axes, rows], cos_sin f32 [n_pos, rope_dim]; None: no
    rotation.  sections: pairs of each axis (one axis: all of them)."""
    if cos_sin is None:
        return None
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin is [n_pos, rope_dim]")
    n = 1 if pos is None or pos.dim() == 1 else pos.shape[0]
    if pos is None or pos.dim() not in (1, 2) or pos.shape[-1] != rows:
        raise ValueError("pos is [rows] or [axes, rows]")
    n_pos, dim = cos_sin.shape
    sections = (dim // 2,) if sections is None else sections
    if len(sections) != n or n > 3:
        raise ValueError("sections gives the pairs of each of pos's one to three axes")
    sec = (*sections, 0, 0)
    return _ROPE.pack(dim, n, sec[0], sec[1], sec[2], _need(pos, "pos", _i32, n * rows, dev),
                      _need(cos_sin, "cos_sin", _f32, None, dev), n_pos)


def rope_axes(x, pos, cos_sin, sections: Optional[Sequence[int]] = None, out=None, d_status=None, stream=None):
    """x bf16 [rows, heads, d] (strided over rows and heads) with its last rope_dim channels turned;
    out may be x.  See csa2p_rope."""
    dev = x.get_device()
    if x.dim() != 3 or x.dtype is not _bf16 or dev < 0 or x.stride(2) != 1:
        raise ValueError("x is a bf16 device tensor [rows, heads, d] with contiguous channels")
    rows, heads, d = x.shape
    sr, sh, _ = x.stride()
    if rows < 2:                                       # a stride over one row or head means nothing
        sr = heads * d
    if heads < 2:
        sh = d
    if out is None:
        out = _empty((rows, heads, d), _bf16, x.device, stream)
        tr, th = heads * d, d
    else:
        if out.shape != x.shape or out.dtype is not _bf16 or out.get_device() != dev or out.stride(2) != 1:
            raise ValueError("out must be like x")
        tr, th = out.stride(0) if rows > 1 else heads * d, out.stride(1) if heads > 1 else d
    st = (_ready or _lib()).csa2p_rope(x.data_ptr(), sr, sh, out.data_ptr(), tr, th, rows, heads, d,
                                       _axes(pos, cos_sin, sections, rows, dev), _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2p_rope", st)
    return out


def paged_write(cache: PagedCache, x, slot, pos=None, cos_sin=None, sections: Optional[Sequence[int]] = None,
                d_status=None, stream=None):
    """Rows of x (bf16 [rows, d], rows may be strided) rotated (when cos_sin is given), quantised in
    the cache's format and stored at slot int32 [rows].  See csa2p_write."""
    dev = cache._on_gpu()
    if x.dim() != 2 or x.dtype is not _bf16 or x.get_device() != dev or x.stride(1) != 1 or x.shape[1] != cache.d:
        raise ValueError("x is a bf16 tensor [rows, d] on the cache's device with contiguous channels")
    rows = x.shape[0]
    st = (_ready or _lib()).csa2p_write(cache.packed, x.data_ptr(), x.stride(0) if rows > 1 else cache.d, rows,
                                        _need(slot, "slot", _i32, rows, dev), _axes(pos, cos_sin, sections, rows, dev),
                                        _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2p_write", st)


def paged_read(cache: PagedCache, slot, out=None, d_status=None, stream=None):
    """bf16 [rows, d]: the cache rows of slot int32 [rows]; rows of a slot below 0 stay as they were
    (uninitialised in a new `out`).  See csa2p_read."""
    dev = cache._on_gpu()
    rows, d = slot.shape[0], cache.d
    if out is None:
        out, ldo = _empty((rows, d), _bf16, cache.device, stream), d
    else:
        if out.dtype is not _bf16 or out.get_device() != dev or out.shape != (rows, d) or out.stride(1) != 1:
            raise ValueError("out is a bf16 tensor [rows, d] on the cache's device with contiguous channels")
        ldo = out.stride(0) if rows > 1 else d
    st = (_ready or _lib()).csa2p_read(cache.packed, _need(slot, "slot", _i32, rows, dev), rows, out.data_ptr(), ldo,
                                       _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2p_read", st)
    return out


def paged_attn(q, cache: PagedCache, block_table, lens, cu, pos0=None, d_v: Optional[int] = None, window: int = 0,
               ratio_m: int = 1, kv_start=None, sm_scale: Optional[float] = None, out=None, lse=None,
               want_lse: bool = True, workspace=None, d_status=None, stream=None):
    """Attention of new tokens over their requests' pages -> (out bf16 [n_tokens, heads, d_v],
    lse f32 [n_tokens, heads] or None).  q bf16 [n_tokens, heads, d]; block_table int32 [batch,
    width]; lens, pos0, kv_start int32 [batch]; cu int32 [batch + 1]; d_v: leading channels that are
    values, at most 512 (None: all d).  Rows of `out` and `lse` outside every request stay as they
    were.  See csa2p_attn."""
    dev, lib = cache._on_gpu(), _ready or _lib()
    if q.dim() != 3 or q.shape[2] != cache.d or block_table.dim() != 2:
        raise ValueError("q is [n_tokens, heads, the cache's d], block_table [batch, width]")
    T, H, d = q.shape
    d_v = d if d_v is None else d_v
    B, W = lens.shape[0], block_table.shape[1]
    a = _ATTN.pack(*cache.fields, B, T, H, d_v, W, window, ratio_m, 1.0 / math.sqrt(d) if sm_scale is None else sm_scale,
                   _need(q, "q", _bf16, None, dev), _need(block_table, "block_table", _i32, B * W, dev),
                   _need(lens, "lens", _i32, B, dev), _need(cu, "cu", _i32, B + 1, dev), _maybe(pos0, "pos0", _i32, B, dev),
                   _maybe(kv_start, "kv_start", _i32, B, dev))
    at_out = _maybe(out, "out", _bf16, T * H * max(d_v, 0), dev)
    if out is None:
        out = _empty((T, H, max(d_v, 0)), _bf16, cache.device, stream)
        at_out = out.data_ptr()
    at_lse = _maybe(lse, "lse", _f32, T * H, dev)
    if lse is None and want_lse:
        lse = _empty((T, H), _f32, cache.device, stream)
        at_lse = lse.data_ptr()
    need = lib.csa2p_attn_workspace_size(a)
    raw = _stream_of(dev, stream)
    at_ws, size = 0, 0
    if workspace is not None:
        at_ws = _need(workspace, "workspace", workspace.dtype, None, dev)
        size = workspace.numel() * workspace.element_size()
    elif need:
        workspace = _empty(need, torch.uint8, cache.device, stream)
        at_ws, size = workspace.data_ptr(), need
    st = lib.csa2p_attn(a, at_out, at_lse or None, at_ws or None, size, _status(d_status, dev), raw)
    if st:
        raise Csa2Error("csa2p_attn", st)
    return out, lse
