"""Verification shared out over eight, four, two CTAs a request, and one: the choice falls with the batch.  Requests without
nodes fill the batch, so that a few rows stand for all of it."""
import numpy as np
import pytest
import torch

from test_gpu_draft import DEV, F, VerifyCase

pytestmark = pytest.mark.gpu


def batch_of(ctas):
    """The most requests that get so many CTAs each (two a multiprocessor in all)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * sms // ctas if ctas > 1 else 2 * sms + 1


def spread(sizes, B):
    """The given requests at both ends and in the middle of a batch of B."""
    out = [0] * B
    for i, n in enumerate(sizes):
        out[i * (B - 1) // max(len(sizes) - 1, 1)] = n
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("ctas", [8, 4, 2, 1])
@pytest.mark.parametrize("V", [20000, 20003])
def test_every_share(V, ctas, drawn, dtype):
    for near, seed in ((0.5, 70), (4.0, 71)):
        VerifyCase(spread([2, 9, 1, 12, 5], batch_of(ctas)), V, dtype, drawn, "tree", near, seed).check(12)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("V", [1 << 18, (1 << 18) - 3])
def test_one_cta_over_the_largest_vocabulary(V, first, dtype):
    # a lane's sums at their largest: every weight is 1, whole or what is left beside a q of nothing
    c = VerifyCase(spread([1, 3, 1], batch_of(1)), V, dtype, seed=72, shape="star")
    c.p[:] = 1.0
    c.q[:] = 0.0
    c.p[4] = torch.from_numpy(np.random.default_rng(73).random(V).astype(F)).to(dtype)
    c.r[:] = [0.0, 1.0 - 2.0 ** -24][first]
    c.r[len(c.r) // 2] = 0.37
    row = (V + 8) // 8 * 8 if first == 0 else V + 1
    wide = [torch.full((5, row + first), float("nan"), dtype=dtype, device=DEV)[:, first:first + V] for _ in range(2)]
    wide[0].copy_(c.p), wide[1].copy_(c.q)
    c.u[:] = 1.0
    c.q[1] = 2.0
    wide[1].copy_(c.q)                                                     # both children are turned down: 1 - 2, then the row itself
    c.check(3, p=wide[0], q=wide[1])
    c.q[1] = 0.0
    c.p[1, [int(t) for t in c.token[2:4]]] = 0.0                           # turned down, with nothing taken away
    wide[0].copy_(c.p), wide[1].copy_(c.q)
    c.check(3, p=wide[0], q=wide[1])
    c.q = None
    c.check(3, p=wide[0])
