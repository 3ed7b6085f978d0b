"""Binding of libcsa2.so's calls for drafted tokens and shared pages (include/csa2_draft.h).

As in ``paged``: the helpers check what they are given, allocate outputs with torch and call the C
entry points; work goes to the current CUDA stream (or the one given) of the current device, which
has to be the tensors'.  ``layers.draft_plan``, ``draft_layer`` and ``draft_accept`` string them
together with the paged cache's calls.  Outputs are tensors of their own: three allocations take less
of the host's time than one and its views.
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
from .paged import _bf16, _CACHE, _empty, _f32, _i32, _maybe, _need, _status, _stream_of, CacheArgs, PagedCache

DEV_NO_TOKEN = 0x800
MAX_WORDS, MAX_VOCAB, MAX_CACHES = 32, 1 << 18, 32
REFUSED = -2                      # in Fork.dst: the request was not forked

_P, _I32, _I64, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class TreeArgs(ctypes.Structure):
    """csa2d_tree_args"""
    _fields_ = [("batch", _I32), ("n_tokens", _I32), ("words", _I32), ("parent", _P), ("lens", _P), ("cu", _P), ("pos", _P),
                ("seen", _P)]


class TreeAttnArgs(ctypes.Structure):
    """csa2d_tree_attn_args"""
    _fields_ = [("cache", CacheArgs), ("batch", _I32), ("n_tokens", _I32), ("n_heads", _I32), ("d_v", _I32), ("width", _I32),
                ("window", _I32), ("words", _I32), ("sm_scale", _F), ("q", _P), ("block_table", _P), ("lens", _P), ("cu", _P),
                ("seen", _P), ("pos", _P), ("kv_start", _P)]


class VerifyArgs(ctypes.Structure):
    """csa2d_verify_args"""
    _fields_ = [("batch", _I32), ("n_tokens", _I32), ("vocab", _I32), ("type", _I32), ("max_path", _I32), ("p_row", _I64),
                ("q_row", _I64), ("p", _P), ("q", _P), ("token", _P), ("parent", _P), ("cu", _P), ("u", _P), ("r", _P), ("keep", _P),
                ("path", _P), ("next_token", _P), ("delta", _P), ("pos", _P)]


class CompactArgs(ctypes.Structure):
    """csa2d_compact_args"""
    _fields_ = [("batch", _I32), ("width", _I32), ("max_path", _I32), ("block_table", _P), ("lens", _P), ("cu", _P), ("path", _P),
                ("keep", _P), ("pos", _P), ("delta", _P), ("n_tokens", _I32)]


class ShareArgs(ctypes.Structure):
    """csa2d_share_args"""
    _fields_ = [("batch", _I32), ("page", _I32), ("width", _I32), ("n_pages", _I32), ("free_cap", _I32), ("source", _P), ("ends", _P),
                ("lens", _P), ("block_table", _P), ("shares", _P), ("free_pages", _P), ("n_free", _P), ("src", _P), ("dst", _P),
                ("rows", _P)]


_TREE = struct.Struct("@3i4x5P")                              # csa2d_tree_args
_ATTN = struct.Struct(_CACHE.format + "7if7P")                # csa2d_tree_attn_args
_VERIFY = struct.Struct("@5i4x2q12P")                         # csa2d_verify_args
_COMPACT = struct.Struct("@3i4x7Pi4x")                        # csa2d_compact_args
_SHARE = struct.Struct("@5i4x10P")                            # csa2d_share_args

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = csa2.load()
        S, sz, A = ctypes.c_int, ctypes.c_size_t, _P          # A: an argument structure
        for name, res, args in (
                ("csa2d_tree_plan", S, [A, _P, _P]),
                ("csa2d_tree_attn_workspace_size", sz, [A]),
                ("csa2d_tree_attn", S, [A, _P, _P, _P, sz, _P, _P]),
                ("csa2d_tree_verify", S, [A, _P, _P]),
                ("csa2d_compact", S, [A, A, _I32, _P, _P]),
                ("csa2d_page_fork", S, [A, _P, _P]),
                ("csa2d_page_free", S, [A, _P, _P]),
                ("csa2d_page_copy", S, [A, _I32, _P, _P, _P, _I32, _P, _P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _ready = lib
    return _ready


# ------------------------------------------------------------------------------------------ trees
@dataclass
class TreePlan:
    """Positions and masks of a step's nodes."""
    pos: torch.Tensor         # int32 [n_tokens]; -1: a node of no request
    seen: torch.Tensor        # int32 [n_tokens, words]: bit k % 32 of word k / 32: the request's node k


def tree_plan(parent, lens, cu, max_nodes: int, d_status=None, stream=None, out: Optional[TreePlan] = None) -> TreePlan:
    """Positions and masks of trees: parent int32 [n_tokens] (a lower node of the request, or -1), lens
    int32 [batch] rows held with the nodes', cu int32 [batch + 1].  max_nodes: of one request, at most
    1,024 (it gives the masks' width).  See csa2d_tree_plan."""
    dev, T, B = parent.get_device(), parent.numel(), lens.numel()
    words = -(-max_nodes // 32)
    if not 1 <= words <= MAX_WORDS:
        raise ValueError(f"max_nodes is 1..{32 * MAX_WORDS}, not {max_nodes}")
    if out is None:
        out = TreePlan(_empty(T, _i32, parent.device, stream), _empty((T, words), _i32, parent.device, stream))
        at_pos, at_seen = out.pos.data_ptr(), out.seen.data_ptr()
    else:
        at_pos, at_seen = _need(out.pos, "out.pos", _i32, T, dev), _need(out.seen, "out.seen", _i32, T * words, dev)
    a = _TREE.pack(B, T, words, _need(parent, "parent", _i32, T, dev), _need(lens, "lens", _i32, B, dev), _need(cu, "cu", _i32, B + 1, dev),
                   at_pos, at_seen)
    st = (_ready or _lib()).csa2d_tree_plan(a, _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2d_tree_plan", st)
    return out


def tree_attn(q, cache: PagedCache, block_table, lens, cu, seen, pos=None, d_v: Optional[int] = None, window: int = 0, kv_start=None,
              sm_scale: Optional[float] = None, out=None, lse=None, want_lse: bool = True, workspace=None, d_status=None, stream=None):
    """Attention of trees over their requests' pages -> (out bf16 [n_tokens, heads, d_v], lse f32
    [n_tokens, heads] or None).  q bf16 [n_tokens, heads, d]; seen int32 [n_tokens, words] and pos
    int32 [n_tokens] (needed with a window) from tree_plan; the rest as in paged.paged_attn.  See
    csa2d_tree_attn."""
    dev, lib = cache._on_gpu(), _ready or _lib()
    if q.dim() != 3 or q.shape[2] != cache.d or block_table.dim() != 2 or seen.dim() != 2:
        raise ValueError("q is [n_tokens, heads, the cache's d], block_table [batch, width], seen [n_tokens, words]")
    if window > 0 and pos is None:
        raise ValueError("a window needs the nodes' positions")
    T, H, d = q.shape
    d_v = d if d_v is None else d_v
    B, W, words = lens.numel(), block_table.shape[1], seen.shape[1]
    a = _ATTN.pack(*cache.fields, B, T, H, d_v, W, window, words, 1.0 / math.sqrt(d) if sm_scale is None else sm_scale,
                   _need(q, "q", _bf16, None, dev), _need(block_table, "block_table", _i32, B * W, dev), _need(lens, "lens", _i32, B, dev),
                   _need(cu, "cu", _i32, B + 1, dev), _need(seen, "seen", _i32, T * words, dev), _maybe(pos, "pos", _i32, T, dev),
                   _maybe(kv_start, "kv_start", _i32, B, dev))
    at_out = _maybe(out, "out", _bf16, T * H * max(d_v, 0), dev)
    if out is None:
        out = _empty((T, H, max(d_v, 0)), _bf16, cache.device, stream)
        at_out = out.data_ptr()
    at_lse = _maybe(lse, "lse", _f32, T * H, dev)
    if lse is None and want_lse:
        lse = _empty((T, H), _f32, cache.device, stream)
        at_lse = lse.data_ptr()
    need = lib.csa2d_tree_attn_workspace_size(a)
    raw = _stream_of(dev, stream)
    at_ws, size = 0, 0
    if workspace is not None:
        at_ws = _need(workspace, "workspace", workspace.dtype, None, dev)
        size = workspace.numel() * workspace.element_size()
    elif need:
        workspace = _empty(need, torch.uint8, cache.device, stream)
        at_ws, size = workspace.data_ptr(), need
    st = lib.csa2d_tree_attn(a, at_out, at_lse or None, at_ws or None, size, _status(d_status, dev), raw)
    if st:
        raise Csa2Error("csa2d_tree_attn", st)
    return out, lse


@dataclass
class Verdict:
    """What csa2d_tree_verify says of each request (int32 tensors)."""
    keep: torch.Tensor        # [batch] nodes that stay, node 0 among them
    path: torch.Tensor        # [batch, max_path] these nodes; -1 behind them
    token: torch.Tensor       # [batch] the token that follows them
    delta: torch.Tensor       # [batch] keep - nodes: for page_plan


def _rows(t, name: str, T: int, V: int, dtype, dev: int):
    """Address and row stride of probabilities [T, V]."""
    if t.dim() != 2 or t.shape != (T, V) or t.dtype is not dtype or t.get_device() != dev or dev < 0 or (T > 0 and V > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be {dtype} [{T}, {V}] on the GPU with contiguous rows, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr(), t.stride(0) if T > 1 else V


def tree_verify(p, token, parent, cu, u, r, q=None, max_path: Optional[int] = None, d_status=None, stream=None,
                out: Optional[Verdict] = None, pos=None) -> Verdict:
    """Which drafts stay, and the token behind them.  p [n_tokens, vocab] (float32, float16 or bfloat16;
    rows may be strided): the target's probabilities after each node; q like p: those that each node's
    children were drawn from (None: the drafts are certain); token, parent int32 and u f32 [n_tokens];
    cu int32 [batch + 1]; r f32 [batch]; u and r uniform from 0 to 1.  max_path: entries of a path (None:
    n_tokens, at most the 1,024 nodes that a request may have; the trees' largest depth + 1 is enough).  pos int32 [n_tokens]: tree_plan's, so that requests that it left out keep nothing and give
    their nodes' rows back.  See csa2d_tree_verify."""
    dev, T, B = p.get_device(), token.numel(), r.numel()
    if p.dtype not in _TYPES or p.dim() != 2:
        raise ValueError("p is float32, float16 or bfloat16 [n_tokens, vocab]")
    V = p.shape[1]
    max_path = min(max(T, 1), 32 * MAX_WORDS) if max_path is None else max_path
    at_p, p_row = _rows(p, "p", T, V, p.dtype, dev)
    at_q, q_row = (0, V) if q is None else _rows(q, "q", T, V, p.dtype, dev)
    if out is None:
        device = p.device
        out = Verdict(_empty(B, _i32, device, stream), _empty((B, max(max_path, 0)), _i32, device, stream), _empty(B, _i32, device, stream),
                      _empty(B, _i32, device, stream))
        at = (out.keep.data_ptr(), out.path.data_ptr(), out.token.data_ptr(), out.delta.data_ptr())
    else:
        at = (_need(out.keep, "out.keep", _i32, B, dev), _need(out.path, "out.path", _i32, B * max(max_path, 0), dev),
              _need(out.token, "out.token", _i32, B, dev), _need(out.delta, "out.delta", _i32, B, dev))
    a = _VERIFY.pack(B, T, V, _TYPES[p.dtype], max_path, p_row, q_row, at_p, at_q, _need(token, "token", _i32, T, dev),
                     _need(parent, "parent", _i32, T, dev), _need(cu, "cu", _i32, B + 1, dev), _need(u, "u", _f32, T, dev),
                     _need(r, "r", _f32, B, dev), *at, _maybe(pos, "pos", _i32, T, dev))
    st = (_ready or _lib()).csa2d_tree_verify(a, _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2d_tree_verify", st)
    return out


# ------------------------------------------------------------------------------------------ pages
def _sets(caches: Sequence[PagedCache]):
    """(device, [(packed caches, how many)]): as many calls as their number needs."""
    if not caches:
        raise ValueError("no cache is given")
    dev = caches[0]._on_gpu()
    for c in caches:
        if c.index != dev:
            raise ValueError("the caches are on several devices")
    if len(caches) <= MAX_CACHES:
        return dev, ((b"".join([c.packed for c in caches]), len(caches)),)
    parts = [caches[i:i + MAX_CACHES] for i in range(0, len(caches), MAX_CACHES)]
    return dev, [(b"".join(c.packed for c in part), len(part)) for part in parts]


def paged_compact(caches: Sequence[PagedCache], block_table, lens, cu, path, keep, d_status=None, stream=None, pos=None, delta=None):
    """Rows base + path[b][i] of each request's nodes moved to base + i, i < keep[b], in every cache (base
    = lens[b] - nodes).  block_table int32 [batch, width], lens and keep int32 [batch], cu int32 [batch +
    1], path int32 [batch, max_path].  pos int32 [n_tokens]: tree_plan's, so that requests that it left out
    move nothing; delta int32 [batch]: tree_verify's, lowered to take all nodes' rows back where a
    request is left out or its path is refused.  See csa2d_compact."""
    dev, sets = _sets(caches)
    B = lens.numel()
    if block_table.dim() != 2 or path.dim() != 2:
        raise ValueError("block_table is [batch, width], path [batch, max_path]")
    page = caches[0].page
    for c in caches:
        if c.page != page:
            raise ValueError("the caches have pages of several sizes")
    W, L = block_table.shape[1], path.shape[1]
    a = _COMPACT.pack(B, W, L, _need(block_table, "block_table", _i32, B * W, dev), _need(lens, "lens", _i32, B, dev),
                      _need(cu, "cu", _i32, B + 1, dev), _need(path, "path", _i32, B * L, dev), _need(keep, "keep", _i32, B, dev),
                      _maybe(pos, "pos", _i32, None, dev), _maybe(delta, "delta", _i32, B, dev), 0 if pos is None else pos.numel())
    status, raw = _status(d_status, dev), _stream_of(dev, stream)
    for packed, n in sets:
        st = (_ready or _lib()).csa2d_compact(a, packed, n, status, raw)
        if st:
            raise Csa2Error("csa2d_compact", st)


@dataclass
class Fork:
    """The pages whose contents a fork has to copy (int32 [batch] each): see page_copy."""
    src: torch.Tensor         # -1: none
    dst: torch.Tensor         # -1: none; REFUSED: the request was not forked
    rows: torch.Tensor


def _share(which, name: str, lens, block_table, shares, free_pages, n_free, page: int, fork, out):
    dev, B = lens.get_device(), lens.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table is [batch, width]")
    W = block_table.shape[1]
    at = _need(which, name, _i32, B, dev)
    return dev, _SHARE.pack(B, page, W, shares.numel(), free_pages.numel(), at if fork else 0, 0 if fork else at,
                            _need(lens, "lens", _i32, B, dev), _need(block_table, "block_table", _i32, B * W, dev),
                            _need(shares, "shares", _i32, None, dev), _need(free_pages, "free_pages", _i32, None, dev),
                            _need(n_free, "n_free", _i32, 1, dev), *out)


def page_fork(source, lens, block_table, shares, free_pages, n_free, page: int, d_status=None, stream=None,
              out: Optional[Fork] = None) -> Fork:
    """Requests with source[b] >= 0 take over that request's rows: lens, block_table, shares (int32
    [n_pages], a page's holders beyond the first) and n_free are updated, and the pages to copy are
    returned.  From then on such requests end with page_free: page_plan gives pages back without looking at
    shares, so it may take rows of them back only down to the length at the fork.  See csa2d_page_fork."""
    B, dev = lens.numel(), lens.get_device()
    if out is None:
        device = lens.device
        out = Fork(_empty(B, _i32, device, stream), _empty(B, _i32, device, stream), _empty(B, _i32, device, stream))
        at = (out.src.data_ptr(), out.dst.data_ptr(), out.rows.data_ptr())
    else:
        at = (_need(out.src, "out.src", _i32, B, dev), _need(out.dst, "out.dst", _i32, B, dev), _need(out.rows, "out.rows", _i32, B, dev))
    dev, a = _share(source, "source", lens, block_table, shares, free_pages, n_free, page, True, at)
    st = (_ready or _lib()).csa2d_page_fork(a, _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2d_page_fork", st)
    return out


def page_free(ends, lens, block_table, shares, free_pages, n_free, page: int, d_status=None, stream=None):
    """Requests with ends[b] != 0 end: their pages lose a holder, and those without one go on the free
    list; lens, shares, free_pages and n_free are updated.  See csa2d_page_free."""
    dev, a = _share(ends, "ends", lens, block_table, shares, free_pages, n_free, page, False, (0, 0, 0))
    st = (_ready or _lib()).csa2d_page_free(a, _status(d_status, dev), _stream_of(dev, stream))
    if st:
        raise Csa2Error("csa2d_page_free", st)


def page_copy(caches: Sequence[PagedCache], src, dst, rows=None, d_status=None, stream=None):
    """In every cache the first rows[i] rows (None: all) of page src[i] copied to page dst[i]; pairs with
    a page below 0 are skipped.  int32 [n] each.  See csa2d_page_copy."""
    dev, sets = _sets(caches)
    n = src.numel()
    at = _need(src, "src", _i32, n, dev), _need(dst, "dst", _i32, n, dev), _maybe(rows, "rows", _i32, n, dev) or None
    status, raw = _status(d_status, dev), _stream_of(dev, stream)
    for packed, k in sets:
        st = (_ready or _lib()).csa2d_page_copy(packed, k, *at, n, status, raw)
        if st:
            raise Csa2Error("csa2d_page_copy", st)
