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
