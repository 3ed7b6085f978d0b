"""Paged-cache calls that are refused on the host, or answered there: nothing here reaches the GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from fp4_kv_cache_gb300 import paged
from test_paged_host import FAKE, INVALID, ROOT, attn, cache, lib, plan, rope      # noqa: F401

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


# ------------------------------------------------------------------ outputs that overlap
def test_rope_outputs_that_overlap_refused(lib):
    # each stride holds a vector, and still the second head of a row lies on the next row
    f, r, other = lib.csa2p_rope, ctypes.byref(rope()), FAKE + (1 << 30)
    call = lambda rows, heads, row, head, x=FAKE: f(x, row, head, other, row, head, rows, heads, 576, r, None, None)  # noqa: E731
    assert call(4, 2, 576, 576) == INVALID
    assert call(4, 2, 576, 576, other) == INVALID                          # in place
    assert call(4, 3, 1152, 576) == INVALID                                # heads reach the next row
    assert call(4, 2, 576, 4 * 576 - 8) == INVALID                         # rows reach the next head
    assert call(4, 2, 640, 960) == INVALID                                 # head 1 between two rows, on both
    assert call(3, 3, 1 << 60, (1 << 60) + 8) == INVALID                   # far apart, but two by two on each other


def strides(overlapping):
    """(rows, heads, row stride, head stride) of vectors of 16 elements that share elements, or do not."""
    for rows, heads in ((2, 2), (3, 2), (2, 4), (4, 3)):
        for R in range(16, 120, 8):
            for H in range(16, 120, 8):
                at = sorted(r * R + h * H for r in range(rows) for h in range(heads))
                if any(b - a < 16 for a, b in zip(at, at[1:])) == overlapping:
                    yield rows, heads, R, H


def test_rope_overlaps_by_enumeration(lib):
    # (the other strides are accepted, and so run on a GPU only)
    r, n = ctypes.byref(rope(dim=16, sec=(8, 0, 0))), 0
    for rows, heads, R, H in strides(True):
        assert lib.csa2p_rope(FAKE, R, H, FAKE + (1 << 20), R, H, rows, heads, 16, r, None, None) == INVALID, (rows, heads, R, H)
        n += 1
    assert n > 100


# ------------------------------------------------------------------ addresses that hold no 32-bit values
OFF = FAKE + 2


@pytest.mark.parametrize("name", ["lens", "delta", "lens_out", "block_table", "free_pages", "n_free", "n_free_out", "cu",
                                  "slot", "row_req", "row_pos"])
def test_plan_addresses_refused(lib, name):
    assert lib.csa2p_page_plan(plan(**{name: OFF}), None, None) == INVALID


@pytest.mark.parametrize("name", ["block_table", "lens", "cu", "pos0", "kv_start"])
def test_attn_addresses_refused(lib, name):
    assert lib.csa2p_attn(ctypes.byref(attn(**{name: OFF})), FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID


def test_other_addresses_refused(lib):
    c, r, other = ctypes.byref(cache()), ctypes.byref(rope()), FAKE + (1 << 20)
    assert lib.csa2p_write(c, FAKE, 576, 4, OFF, None, None, None) == INVALID
    assert lib.csa2p_read(c, OFF, 4, FAKE, 576, None, None) == INVALID
    assert lib.csa2p_attn(ctypes.byref(attn()), FAKE, OFF, FAKE, 1 << 40, None, None) == INVALID
    for status in (OFF, FAKE + 1):
        assert lib.csa2p_page_plan(plan(), status, None) == INVALID
        assert lib.csa2p_rope(FAKE, 576, 576, other, 576, 576, 4, 1, 576, r, status, None) == INVALID
        assert lib.csa2p_write(c, FAKE, 576, 4, FAKE, None, status, None) == INVALID
        assert lib.csa2p_read(c, FAKE, 4, FAKE, 576, status, None) == INVALID
        assert lib.csa2p_attn(ctypes.byref(attn()), FAKE, FAKE, FAKE, 1 << 40, status, None) == INVALID


# ------------------------------------------------------------------ logit scales
@pytest.mark.parametrize("scale", [2.4e38, 2.9e38, -1.0])
def test_attn_scales_refused(lib, scale):
    # times log2(e) no float is left: 0 x infinity would make NaN of a logit of 0
    assert lib.csa2p_attn(ctypes.byref(attn(sm_scale=scale)), FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID


# ------------------------------------------------------------------ a torch without CUDA
def test_package_imports_without_cuda():
    # layers and paged can be imported, and a cache on the CPU be made, where torch has no CUDA calls
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from fp4_kv_cache_gb300 import layers, paged\n"
            "paged.PagedCache.new(2, 16, 64, device='cpu')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
