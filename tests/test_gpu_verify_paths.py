"""Paths of the verification whose length the caller leaves open: as long as a tree can be, not as the call's tokens."""
import pytest
import torch

from fp4_kv_cache_gb300 import draft
from test_gpu_draft import VerifyCase
from test_gpu_paged import DEV, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,entries", [([3] * 700, 1024), ([1024, 2], 1024), ([400, 400], 800), ([5], 5)])
def test_default_path_is_no_longer_than_a_tree(sizes, entries):
    c = VerifyCase(sizes, 8, seed=60, shape="chain", near=0.0)
    c.u[:] = 0.0                                                           # every draft stays
    v = c.check()
    assert tuple(v.path.shape) == (len(sizes), entries) and v.keep.tolist() == sizes
    assert all(v.path[b, :n].tolist() == list(range(n)) for b, n in enumerate(sizes))


def test_many_requests_take_little():
    c = VerifyCase([1] * 4000, 2, seed=61)
    args = (c.p.to(DEV), ints(c.token), ints(c.parent), ints(c.cu), torch.from_numpy(c.u).to(DEV), torch.from_numpy(c.r).to(DEV))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    v = draft.tree_verify(*args, q=None)
    assert torch.cuda.max_memory_allocated() - before <= 4000 * 1024 * 4 + 4 * 4000 * 4 + 8192
    assert v.keep.tolist() == [1] * 4000
