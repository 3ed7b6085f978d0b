"""What tells verification and compaction which requests the tree plan left out, on the host: every refusal."""
import pytest
import torch

from fp4_kv_cache_gb300 import draft, paged
from test_draft_host import OFF, compact, lib, verify  # noqa: F401
from test_paged_host import INVALID, cache

I32 = torch.int32


def test_refused(lib):  # noqa: F811
    one = (paged.CacheArgs * 1)(cache())
    assert lib.csa2d_tree_verify(verify(pos=OFF), None, None) == INVALID
    for bad in (dict(pos=OFF), dict(delta=OFF), dict(n_tokens=-1)):
        assert lib.csa2d_compact(compact(**bad), one, 1, None, None) == INVALID
    assert lib.csa2d_compact(compact(n_tokens=-1), None, 0, None, None) == 0            # no cache: nothing is done


def test_binding_refuses_shapes_types_and_devices():
    i = lambda *s: torch.zeros(s, dtype=I32)                               # noqa: E731
    c = paged.PagedCache.new(2, 16, 64, device="cpu")
    for more in (dict(pos=i(4)), dict(pos=torch.zeros(4)), dict(delta=i(2)), dict(delta=torch.zeros(1))):
        with pytest.raises(ValueError):
            draft.paged_compact([c], i(1, 1), i(1), i(2), i(1, 1), i(1), **more)
    with pytest.raises(ValueError):
        draft.tree_verify(torch.zeros((4, 9)), i(4), i(4), i(2), torch.zeros(4), torch.zeros(1), pos=i(3))
