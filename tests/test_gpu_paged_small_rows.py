"""Attention over rows of few channels, where some warps of a CTA stage little of a tile: many calls, each with
the same bits and no wait that ran out."""
import pytest
import torch

from fp4_kv_cache_gb300 import draft, paged
from test_gpu_draft import TreeCase, check as check_tree
from test_gpu_paged import AttnCase, DEV, I32, check, ints, status

pytestmark = pytest.mark.gpu
SHAPES = [(32, 8), (64, 64), (96, 96), (128, 128), (256, 256), (288, 264)]


def same_every_time(first, call, n=400):
    st, off = status(), []
    for _ in range(n):
        out, lse = call(st)
        off.append((out.view(torch.int16) != first[0].view(torch.int16)).sum() + (lse.view(I32) != first[1].view(I32)).sum())
    assert int(torch.stack(off).sum()) == 0 and int(st) == 0


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.MXFP8, paged.BF16])
@pytest.mark.parametrize("d,dv", SHAPES)
def test_attn_small_rows_again_and_again(d, dv, fmt):
    c = AttnCase([130 + 2 * b for b in range(31)], [1 + b % 30 for b in range(31)], 128, d, dv, fmt, 64, seed=d)
    first = check(c)
    table, lens, cu = torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu)
    same_every_time(first, lambda st: paged.paged_attn(c.q, c.cache, table, lens, cu, d_v=dv, sm_scale=c.sm, d_status=st))


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.MXFP8, paged.BF16])
@pytest.mark.parametrize("d,dv", SHAPES)
def test_tree_attn_small_rows_again_and_again(d, dv, fmt):
    c = TreeCase([130 + 2 * b for b in range(31)], [1 + b % 30 for b in range(31)], 128, d, dv, fmt, 64, seed=d)
    first = check_tree(c)
    table, lens, cu = torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu)
    seen, pos = torch.from_numpy(c.seen.view("int32")).to(DEV), ints(c.pos)
    same_every_time(first, lambda st: draft.tree_attn(c.q, c.cache, table, lens, cu, seen, pos, d_v=dv, sm_scale=c.sm, d_status=st))
