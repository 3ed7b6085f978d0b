"""Paged-cache calls that are refused on the host, or answered there: nothing here reaches the GPU."""
import ctypes

import pytest
import torch

from fp4_kv_cache_gb300 import paged
from test_paged_host import FAKE, INVALID, attn, cache, lib, plan, rope      # noqa: F401

U8 = torch.uint8


# ------------------------------------------------------------------ pages that overlap
def test_expanded_pages_refused():
    # a page seen n times over (stride 0) is not n dense pages
    codes, scales = torch.zeros((5, 16, 288), dtype=U8), torch.zeros((5, 16, 18), dtype=U8)
    with pytest.raises(ValueError, match="overlap"):
        paged.PagedCache(codes[:1].expand(5, 16, 288), scales)
    with pytest.raises(ValueError, match="overlap"):
        paged.PagedCache(codes, scales[:1].expand(5, 16, 18))
    with pytest.raises(ValueError, match="overlap"):
        paged.PagedCache(torch.zeros((1, 16, 64), dtype=torch.bfloat16).expand(3, 16, 64))
    with pytest.raises(ValueError, match="overlap"):
        paged.PagedCache(torch.as_strided(codes, (5, 16, 288), (8 * 288, 288, 1)), scales)
    # one page has no distance to a next one
    assert paged.PagedCache(codes[:1].expand(1, 16, 288), scales[:1]).fields[-2:] == (0, 0)


# ------------------------------------------------------------------ calls of no rows
def test_no_rows_have_no_positions(lib):
    # a step that only takes rows back: its tensors are empty, and empty tensors have no address
    r, c = ctypes.byref(rope(pos=None)), ctypes.byref(cache())
    assert lib.csa2p_write(c, None, 576, 0, None, r, None, None) == 0
    assert lib.csa2p_rope(None, 1152, 576, None, 1152, 576, 0, 2, 576, r, None, None) == 0
    assert lib.csa2p_write(c, FAKE, 576, 1, FAKE, r, None, None) == INVALID
    bad = ctypes.byref(rope(sec=(31, 0, 0)))                               # still no rotation of 32 pairs
    assert lib.csa2p_write(c, None, 576, 0, None, bad, None, None) == INVALID
    assert lib.csa2p_rope(None, 1152, 576, None, 1152, 576, 0, 2, 576, bad, None, None) == INVALID
