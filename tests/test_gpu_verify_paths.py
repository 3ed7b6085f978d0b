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


def test_a_call_without_tokens_takes_probabilities_of_any_stride():
    # rows that are not there have no layout
    i, f = (lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)), (lambda n: torch.zeros(n, device=DEV))
    for p in (torch.empty((0, 8), device=DEV), torch.empty_strided((0, 8), (1, 0), device=DEV), torch.empty((8, 0), device=DEV).T):
        for q in (None, p):
            v = draft.tree_verify(p, i(0), i(0), i(3), f(0), f(2), q=q)
            assert v.keep.tolist() == v.delta.tolist() == [0, 0] and v.token.tolist() == [-1, -1] and v.path.tolist() == [[-1], [-1]]
    with pytest.raises(ValueError):
        draft.tree_verify(torch.rand((8, 3), device=DEV).T, i(3), i(3), ints([0, 3]), f(3), f(1))
