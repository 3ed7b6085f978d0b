"""Binding of the paged-cache calls of libcsa2.so (include/csa2_paged.h).

As in ``csa2``: the ``csa2p_*`` functions mirror the C entry points, the short-named helpers
allocate outputs with torch and call them, and everything is computed by the library's
kernels.  Work goes to the current CUDA stream of the tensors' device (or the one given).
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import csa2
from .csa2 import _check

MXFP4, NVFP4_E4M3_16, MXFP8, BF16 = 0, 1, 2, 3
DEV_NO_PAGES, DEV_TABLE_FULL, DEV_ROWS = 0x100, 0x200, 0x400
MAX_BATCH = 16384

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


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


_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = csa2.load()
        S, sz = ctypes.c_int, ctypes.c_size_t
        for name, res, args in (
                ("csa2p_page_plan", S, [ctypes.POINTER(PlanArgs), _P, _P]),
                ("csa2p_rope", S, [_P, _I64, _I64, _P, _I64, _I64, _I32, _I32, _I32, ctypes.POINTER(RopeAxes), _P, _P]),
                ("csa2p_write", S, [ctypes.POINTER(CacheArgs), _P, _I64, _I32, _P, ctypes.POINTER(RopeAxes), _P, _P]),
                ("csa2p_read", S, [ctypes.POINTER(CacheArgs), _P, _I32, _P, _I64, _P, _P]),
                ("csa2p_attn_workspace_size", sz, [ctypes.POINTER(AttnArgs)]),
                ("csa2p_attn", S, [ctypes.POINTER(AttnArgs), _P, _P, _P, sz, _P, _P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _ready = lib
    return _ready


def _stream_of(t: torch.Tensor, stream):
    """Raw stream of a call: the one given, else the current one of the tensor's device.  The
    library works on the current device, so that has to be the tensor's."""
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}: make it the current device (torch.cuda.device)")
    return (stream or torch.cuda.current_stream()).cuda_stream


def _need(t: Optional[torch.Tensor], name: str, dtype, shape=None, device=None):
    """Address of a contiguous device tensor of this type (and shape), or None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'the GPU'}, not {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class PagedCache:
    """One layer's pages: codes [n_pages, page, row bytes] uint8 and scales [n_pages, page, scales a
    row] uint8 (told apart by their widths: MXFP4, E2M1 + E4M3/16, or MXFP8), or bf16 values
    [n_pages, page, d] without scales.  Rows are contiguous within a page; pages may lie apart
    (a view of a larger buffer)."""

    def __init__(self, codes: torch.Tensor, scales: Optional[torch.Tensor] = None):
        if codes.dim() != 3 or (scales is not None and (scales.dim() != 3 or scales.shape[:2] != codes.shape[:2])):
            raise ValueError("codes and scales are [n_pages, page, bytes of a row]")
        n, page, w = codes.shape
        if scales is None:
            if codes.dtype != torch.bfloat16:
                raise ValueError("a cache without scales holds bf16 values")
            fmt, d = BF16, w
        else:
            if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or scales.device != codes.device:
                raise ValueError("codes and scales are uint8 tensors on one device")
            ratio = w / scales.shape[2] if scales.shape[2] else 0
            try:
                fmt = {16: MXFP4, 8: NVFP4_E4M3_16, 32: MXFP8}[ratio]
            except KeyError:
                raise ValueError("the widths of codes and scales fit no row format") from None
            d = w if fmt == MXFP8 else 2 * w
        for t in (codes, scales):
            if t is not None and not (t.stride(2) == 1 and t.stride(1) == t.shape[2]):
                raise ValueError("rows must be contiguous within a page")
        self.codes, self.scales, self.fmt, self.d, self.page, self.n_pages = codes, scales, fmt, d, page, n
        self.device = codes.device
        self.args = CacheArgs(fmt, d, page, n, codes.data_ptr(), scales.data_ptr() if scales is not None else None,
                              codes.stride(0) * codes.element_size() if n > 1 else 0,
                              scales.stride(0) if scales is not None and n > 1 else 0)

    def _on_gpu(self):
        if not self.codes.is_cuda:
            raise ValueError("libcsa2 takes device tensors (got a CPU cache)")

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


def csa2p_page_plan(args: PlanArgs, d_status=None, stream: int = 0):
    _check("csa2p_page_plan", _lib().csa2p_page_plan(ctypes.byref(args), d_status, stream))


def page_plan(lens, delta, block_table, free_pages, n_free, page: int, n_rows: int, in_place: bool = False,
              plan: Optional[PagePlan] = None, d_status=None, stream=None) -> PagePlan:
    """One step of the requests' bookkeeping: block_table [batch, width] and free_pages are updated,
    the rest is returned (into `plan`'s tensors when given).  in_place: lens and n_free are
    overwritten with the new lengths and the new count, as a captured graph needs it."""
    dev, B = lens.device, lens.shape[0]
    if plan is None:
        buf = torch.empty(2 * B + 2 + 3 * n_rows, dtype=torch.int32, device=dev)
        o = 2 * B + 2
        plan = PagePlan(lens if in_place else buf[:B], buf[B:2 * B + 1], buf[o:o + n_rows], buf[o + n_rows:o + 2 * n_rows],
                        buf[o + 2 * n_rows:], n_free if in_place else buf[2 * B + 1:o])
    i32 = torch.int32
    a = PlanArgs(B, page, block_table.shape[1], free_pages.shape[0], n_rows, _need(lens, "lens", i32, (B,), dev),
                 _need(delta, "delta", i32, (B,), dev), _need(plan.lens, "plan.lens", i32, (B,), dev),
                 _need(block_table, "block_table", i32, (B, block_table.shape[1]), dev),
                 _need(free_pages, "free_pages", i32, (free_pages.shape[0],), dev), _need(n_free, "n_free", i32, (1,), dev),
                 _need(plan.n_free, "plan.n_free", i32, (1,), dev), _need(plan.cu, "plan.cu", i32, (B + 1,), dev),
                 _need(plan.slot, "plan.slot", i32, (n_rows,), dev), _need(plan.row_req, "plan.row_req", i32, (n_rows,), dev),
                 _need(plan.row_pos, "plan.row_pos", i32, (n_rows,), dev))
    csa2p_page_plan(a, _need(d_status, "d_status", i32, None, dev), _stream_of(lens, stream))
    return plan


def _axes(pos, cos_sin, sections, rows: int, dev) -> Optional[RopeAxes]:
    """csa2p_rope_axes of pos int32 [rows] or [axes, rows], cos_sin f32 [n_pos, rope_dim]; None: no
    rotation.  sections: pairs of each axis (one axis: all of them)."""
    if cos_sin is None:
        return None
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin is [n_pos, rope_dim]")
    if pos is None or pos.shape[-1] != rows or pos.dim() not in (1, 2):
        raise ValueError("pos is [rows] or [axes, rows]")
    n = pos.shape[0] if pos.dim() == 2 else 1
    sections = [cos_sin.shape[1] // 2] if sections is None else sections
    if len(sections) != n or n > 3:
        raise ValueError("sections gives the pairs of each of pos's one to three axes")
    return RopeAxes(cos_sin.shape[1], n, (_I32 * 3)(*sections), _need(pos, "pos", torch.int32, None, dev),
                    _need(cos_sin, "cos_sin", torch.float32, None, dev), cos_sin.shape[0])


def rope_axes(x, pos, cos_sin, sections: Optional[Sequence[int]] = None, out=None, d_status=None, stream=None):
    """x bf16 [rows, heads, d] (strided over rows and heads) with its last rope_dim channels turned;
    out may be x.  See csa2p_rope."""
    if x.dim() != 3 or x.dtype != torch.bfloat16 or not x.is_cuda or x.stride(2) != 1:
        raise ValueError("x is a bf16 device tensor [rows, heads, d] with contiguous channels")
    rows, heads, d = x.shape
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or out.stride(2) != 1:
        raise ValueError("out must be like x")
    r = _axes(pos, cos_sin, sections, rows, x.device)
    # a stride over one row or one head only means nothing: the dense one stands in for it
    strides = [(t.stride(0) if rows > 1 else heads * d, t.stride(1) if heads > 1 else d) for t in (x, out)]
    _check("csa2p_rope", _lib().csa2p_rope(
        x.data_ptr(), *strides[0], out.data_ptr(), *strides[1], rows, heads, d,
        ctypes.byref(r) if r is not None else None, _need(d_status, "d_status", torch.int32, None, x.device),
        _stream_of(x, stream)))
    return out


def paged_write(cache: PagedCache, x, slot, pos=None, cos_sin=None, sections: Optional[Sequence[int]] = None,
                d_status=None, stream=None):
    """Rows of x (bf16 [rows, d], rows may be strided) rotated (when cos_sin is given), quantised in
    the cache's format and stored at slot int32 [rows].  See csa2p_write."""
    cache._on_gpu()
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.device != cache.device or x.stride(1) != 1 or x.shape[1] != cache.d:
        raise ValueError("x is a bf16 tensor [rows, d] on the cache's device with contiguous channels")
    rows = x.shape[0]
    r = _axes(pos, cos_sin, sections, rows, x.device)
    _check("csa2p_write", _lib().csa2p_write(
        ctypes.byref(cache.args), x.data_ptr(), x.stride(0) if rows > 1 else cache.d, rows,
        _need(slot, "slot", torch.int32, (rows,), x.device), ctypes.byref(r) if r is not None else None,
        _need(d_status, "d_status", torch.int32, None, x.device), _stream_of(x, stream)))


def paged_read(cache: PagedCache, slot, out=None, d_status=None, stream=None):
    """bf16 [rows, d]: the cache rows of slot int32 [rows]; rows of a slot below 0 stay as they were
    (uninitialised in a new `out`).  See csa2p_read."""
    cache._on_gpu()
    rows = slot.shape[0]
    if out is None:
        out = torch.empty((rows, cache.d), dtype=torch.bfloat16, device=cache.device)
    if out.dtype != torch.bfloat16 or out.device != cache.device or out.shape != (rows, cache.d) or out.stride(1) != 1:
        raise ValueError("out is a bf16 tensor [rows, d] on the cache's device with contiguous channels")
    _check("csa2p_read", _lib().csa2p_read(
        ctypes.byref(cache.args), _need(slot, "slot", torch.int32, (rows,), cache.device), rows, out.data_ptr(),
        out.stride(0) if rows > 1 else cache.d, _need(d_status, "d_status", torch.int32, None, cache.device),
        _stream_of(out, stream)))
    return out


def paged_attn(q, cache: PagedCache, block_table, lens, cu, pos0=None, d_v: Optional[int] = None, window: int = 0,
               ratio_m: int = 1, kv_start=None, sm_scale: Optional[float] = None, out=None, lse=None,
               want_lse: bool = True, workspace=None, d_status=None, stream=None):
    """Attention of new tokens over their requests' pages -> (out bf16 [n_tokens, heads, d_v],
    lse f32 [n_tokens, heads] or None).  q bf16 [n_tokens, heads, d]; block_table int32 [batch,
    width]; lens, pos0, kv_start int32 [batch]; cu int32 [batch + 1].  Rows of `out` and `lse`
    outside every request stay as they were.  See csa2p_attn."""
    cache._on_gpu()
    dev, lib, i32 = cache.device, _lib(), torch.int32
    if q.dim() != 3 or q.shape[2] != cache.d:
        raise ValueError("q is [n_tokens, heads, the cache's d]")
    T, H, d = q.shape
    d_v = d if d_v is None else d_v
    B = lens.shape[0]
    if block_table.dim() != 2:
        raise ValueError("block_table is [batch, width]")
    W = block_table.shape[1]
    a = AttnArgs(cache.args, B, T, H, d_v, W, window, ratio_m, 1.0 / math.sqrt(d) if sm_scale is None else sm_scale,
                 _need(q, "q", torch.bfloat16, None, dev), _need(block_table, "block_table", i32, (B, W), dev),
                 _need(lens, "lens", i32, (B,), dev), _need(cu, "cu", i32, (B + 1,), dev), _need(pos0, "pos0", i32, (B,), dev),
                 _need(kv_start, "kv_start", i32, (B,), dev))
    if out is None:
        out = torch.empty((T, H, max(d_v, 0)), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    ref = ctypes.byref(a)
    need = lib.csa2p_attn_workspace_size(ref)
    raw = _stream_of(q, stream)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if stream is not None:
            workspace.record_stream(stream)
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("csa2p_attn", lib.csa2p_attn(
        ref, _need(out, "out", torch.bfloat16, (T, H, d_v), dev), _need(lse, "lse", torch.float32, (T, H), dev),
        workspace.data_ptr() if workspace is not None else None, size, _need(d_status, "d_status", i32, None, dev), raw))
    return out, lse
