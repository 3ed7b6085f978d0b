"""Paged-cache calls that are refused on the host, or answered there: nothing here reaches the GPU."""
import pytest
import torch

from fp4_kv_cache_gb300 import paged

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
