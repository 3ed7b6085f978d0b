"""Paged-cache calls at their edges: steps after a shortage of pages, offsets that step down or leave
the queries, masks that leave leading pages unread, rows that are not finite, calls at once."""
import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_gb300 import csa2, layers, paged
from test_gpu_paged import AttnCase, DEV, FMTS, I32, check, close, cos_sin, ints, status, turned32, values64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ offsets of the queries
@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("cu", [[0, 5, 0, 5], [0, 3, 1, 5], [0, 3, 1, 2], [5, 0, 5, 5], [0, 7, 4, 9], [2, -1, 3, 5]])
def test_attn_offsets_that_step_down(H, cu):
    # two requests would write the same rows: flagged, nothing written, whatever the tiles come to
    c = AttnCase([40, 7, 33], [5, 0, 0], H, 128, 128, paged.MXFP4, 32, seed=21)
    c.cu = np.array(cu)
    out = torch.full((5, H, 128), 3.0, device=DEV).bfloat16()
    lse, st = torch.full((5, H), 3.0, device=DEV), status()
    c.run(st, out=out, lse=lse)
    assert int(st) == csa2.DEV_BAD_INDEX
    assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


@pytest.mark.parametrize("cu", [[-3, -7, 0, 5], [0, 5, 900, 30], [0, 0, 5, 5], [-9, 0, 5, 700]])
def test_attn_offsets_outside_do_not_step_down(cu):
    # held to 0..n_tokens these offsets do not decrease: the one request inside is done
    c = AttnCase([40, 37, 33], [5, 0, 0], 16, 128, 128, paged.MXFP4, 32, pos0=[35, 32, 28], seed=22)
    c.cu = np.clip(cu, 0, 5)
    want, _ = check(c)
    c.cu, st = np.array(cu), status()
    got, _ = c.run(st)
    assert torch.equal(got, want) and int(st) == 0


@pytest.mark.parametrize("front,back", [(0, 4), (4, 0), (3, 5)])
@pytest.mark.parametrize("window,ratio,pos0", [(0, 1, None), (5, 1, None), (0, 1, [97, 46]), (7, 2, [180, 100])])
def test_attn_queries_cut_off(front, back, window, ratio, pos0):
    # offsets that reach past q at either end: the tokens that q holds keep their positions
    c = AttnCase([100, 60], [7, 10], 16, 128, 128, paged.MXFP4, 16, window, ratio, pos0, seed=23)
    o, l, ob, lb = c.ref()
    keep = slice(front, 17 - back)
    c.q, c.cu, st = c.q[keep].contiguous(), c.cu - front, status()
    out, lse = c.run(st)
    close(out, o[keep], ob[keep])
    close(lse, l[keep], lb[keep])
    assert int(st) == 0


def test_layer_with_more_rows_than_it_is_given():
    # a step of ten new rows, six of them given: flagged, and the six attend what they would have
    H, d, page, fmt = 16, 128, 16, paged.MXFP8
    g = torch.Generator(device=DEV).manual_seed(5)
    x, q = torch.randn((30, d), generator=g, device=DEV).bfloat16(), torch.randn((30, H, d), generator=g, device=DEV).bfloat16()
    cs, got = cos_sin(100, 32), []
    for T in (10, 6):
        cache = paged.PagedCache.new(8, page, d, fmt)
        cache.scales.fill_(127)
        state = layers.PagedState(ints([0]), ints([[-1] * 4]), ints(range(8)), ints([8]))
        layers.paged_layer(cache, state, layers.PagedInput(q[:20], x[:20], ints([20]), cs), d_v=128)
        cache.codes[int(state.block_table[0, 1]), 4:] = 0x70     # what the page held before: not to be seen
        st = status()
        got.append(layers.paged_layer(cache, state, layers.PagedInput(q[20:20 + T], x[20:20 + T], ints([10]), cs), d_v=128, d_status=st))
        assert int(st) == (0 if T == 10 else paged.DEV_ROWS)
    assert torch.equal(got[1].out, got[0].out[:6]) and torch.equal(got[1].lse, got[0].lse[:6])
