"""Requests that the plan of a step of drafts leaves out: one rule for the attention, the verification and the rows that
stay, so that such a request is afterwards as it was before the step."""
import numpy as np
import pytest
import torch

from fp4_kv_cache_gb300 import csa2, draft, layers, paged
from test_gpu_draft import VerifyCase, bytes_cache, compact_ref, random_tree, raw, table_of, verify_ref
from test_gpu_paged import DEV, I32, cos_sin, ints, status

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ verification
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("sizes,V", [([9, 40, 1, 0, 7], 60), ([5, 6, 7], 40000), ([2] * 300, 33)])
def test_verify_leaves_out_what_the_plan_left_out(sizes, V, drawn):
    c = VerifyCase(sizes, V, drawn=drawn, near=0.3, seed=50)
    pos = torch.arange(sum(sizes), dtype=I32, device=DEV)
    for out in ([], [1], [0, 2], range(len(sizes))):
        pos[:] = 5
        for b in out:
            pos[c.cu[b]:c.cu[b + 1]] = -1
        st = status()
        v = draft.tree_verify(c.p.to(DEV), ints(c.token), ints(c.parent), ints(c.cu), torch.from_numpy(c.u).to(DEV), torch.from_numpy(c.r).to(DEV),
                              q=None if c.q is None else c.q.to(DEV), max_path=12, d_status=st, pos=pos)
        keep, path, token, delta, _ = verify_ref(c.p.numpy(), c.q.numpy() if drawn else None, c.token, c.parent, c.cu, c.u, c.r, 12)
        some = False
        for b in out:
            if sizes[b]:
                keep[b], path[b], token[b], delta[b], some = 0, [-1] * 12, -1, -sizes[b], True
        assert v.keep.tolist() == keep and v.path.tolist() == path and v.token.tolist() == token and v.delta.tolist() == delta
        assert int(st) == (csa2.DEV_BAD_INDEX if some else 0)


def test_verify_gives_back_nodes_out_of_range():
    c = VerifyCase([9, 4, 7, 1100], 20, near=0.1, seed=51, pad=3)
    pos = ints([4] * len(c.token))
    args = [c.p.to(DEV), ints(c.token), ints(c.parent), None, torch.from_numpy(c.u).to(DEV), torch.from_numpy(c.r).to(DEV)]
    for cu, want in (([0, 9, 13, 20, 1120], [None, None, None, -1100]), ([-1, 9, 13, 20, 1130], [-10, None, None, -1110]),
                     ([0, 2**31 - 1, 9, 13, 20], [-(2**31 - 1), 0, None, None]), ([-2**31, 2**31 - 1, 9, 9, 9], [-(2**31 - 1), 0, 0, 0])):
        args[3], st = ints(cu), status()
        v = draft.tree_verify(*args, q=c.q.to(DEV), max_path=4, d_status=st, pos=pos)
        assert int(st) == csa2.DEV_BAD_INDEX
        for b, w in enumerate(want):
            if w is None:
                assert int(v.keep[b]) >= 1 and int(v.delta[b]) == int(v.keep[b]) - (cu[b + 1] - cu[b])
            else:
                assert (int(v.keep[b]), int(v.token[b]), int(v.delta[b])) == (0, -1, w) and v.path[b].tolist() == [-1] * 4


# ------------------------------------------------------------------ rows that stay
def test_compact_gives_back_what_does_not_move():
    page, n_pages, width = 8, 60, 5
    r = np.random.default_rng(4)
    #        fine, left out, not rising, past the nodes, keep too large, keep below 0, kept nothing, no nodes, fewer rows, past pos
    lens = [30, 30, 30, 30, 30, 30, 30, 30, 3, 30, 30]
    sizes = [20, 20, 20, 20, 20, 20, 20, 0, 5, 20, 20]
    table, _ = table_of(r, lens, page, n_pages, width)
    path = np.tile(np.array([0, 3, 4, 9, 19]), (11, 1))
    path[2, 2], path[3, 4] = 3, 20
    keep = [5, 5, 5, 5, 6, -1, 0, 0, 2, 3, 4]
    cu = np.cumsum([0] + sizes).tolist()
    n_tokens = cu[10]                                                       # the last request's nodes are not all there
    pos = ints([7] * n_tokens)
    pos[cu[1]:cu[2]] = -1
    delta0 = [-15, -15, 3, -30, -20, -19, 0, 7, -3, -30, -17]               # (-30: the request ends, whatever stays)
    want_delta = [-15, -20, -20, -30, -20, -20, 0, 7, -3, -30, -20]
    for caches in ([bytes_cache(n_pages, page, 64, paged.MXFP4, 5)], [bytes_cache(n_pages, page, 32, paged.BF16, i) for i in range(35)]):
        before, st, delta = [raw(c) for c in caches], status(), ints(delta0)
        draft.paged_compact(caches, ints(table), ints(lens), ints(cu), ints(path), ints(keep), d_status=st, pos=pos, delta=delta)
        moved = list(keep)
        moved[1] = moved[10] = 0
        for c, want in zip(caches, before):
            compact_ref(want, table, lens, cu, path, moved, page, n_pages)
            assert all(np.array_equal(a, b) for a, b in zip(raw(c), want))
        assert int(st) == csa2.DEV_BAD_INDEX and delta.tolist() == want_delta


def test_compact_delta_alone():
    # without pos nothing is left out; a request that keeps nothing is no mistake: its delta is the server's
    page, table = 8, np.array([[0, 1], [2, 3], [4, 5]])
    cache, st, delta = bytes_cache(6, page, 64, paged.MXFP8, 5), status(), ints([-4, 0, 5])
    want = raw(cache)
    args = (table, [14, 16, 9], [0, 6, 10, 10], np.array([[0, 2], [-1, -1], [-1, -1]]), [2, 0, 0])
    compact_ref(want, *args, page, 6)
    draft.paged_compact([cache], *(ints(a) for a in args), d_status=st, delta=delta)
    assert int(st) == 0 and delta.tolist() == [-4, 0, 5] and all(np.array_equal(a, b) for a, b in zip(raw(cache), want))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("case", ["more nodes than max_nodes", "more nodes than any call takes", "nodes past the inputs' rows"])
def test_a_step_leaves_out_what_its_plan_left_out(case, given):
    """One tree is larger than the step takes: its request has the rows and pages of before, the others go on.  The
    verification may know the plan's positions or not: what stays is the same."""
    H, d, page, W, B, V, fmt = 4, 64, 16, 90, 3, 41, paged.MXFP4
    r, g = np.random.default_rng(3), torch.Generator(device=DEV).manual_seed(3)
    cs = cos_sin(1600, 32)
    caches = [paged.PagedCache.new(200, page, d, fmt) for _ in range(2)]
    state = layers.PagedState(ints([0] * B), ints(np.full((B, W), -1)), ints(range(200)), ints([200]))

    def inputs(delta, n=None):
        n = sum(delta) if n is None else n
        return layers.PagedInput(torch.randn((n, H, d), generator=g, device=DEV).bfloat16(), torch.randn((n, d), generator=g, device=DEV).bfloat16(),
                                 ints(delta), cs)

    first = layers.paged_layer(caches[0], state, inputs([50, 33, 70]), 0, d)
    layers.paged_layer_again(caches[1], state, inputs([50, 33, 70]), first.plan, 0, d)
    sizes, max_nodes, bad = {"more nodes than max_nodes": ([12, 40, 5], 32, 1), "more nodes than any call takes": ([12, 1030, 5], 1024, 1),
                             "nodes past the inputs' rows": ([12, 9, 20], 32, 2)}[case]
    T = sum(sizes) - (3 if bad == 2 else 0)
    n_free = int(state.n_free)
    old = [[x[state.block_table[bad, :-(-int(state.lens[bad]) // page)].cpu().numpy()].reshape(-1, x.shape[2])[:int(state.lens[bad])] for x in raw(c)]
           for c in caches]
    before = state.lens.tolist()
    parent = [p for n in sizes for p in random_tree(r, n)][:T]
    st = status()
    step = layers.draft_plan(page, state, inputs(sizes, T), ints(parent), max_nodes, d_status=st)
    for c in caches:
        layers.draft_layer(c, state, inputs(sizes, T), step, 0, d, d_status=st)
    p = torch.softmax(torch.randn((T, V), generator=g, device=DEV), 1)
    q = torch.softmax(torch.randn((T, V), generator=g, device=DEV), 1)
    q[:, 0] = p[:, 0] = 0.5                                                 # drafts of token 0 stay with u below 1
    token, u = torch.zeros(T, dtype=I32, device=DEV), torch.full((T,), 0.25, device=DEV)
    v = draft.tree_verify(p, token, ints(parent), step.plan.cu, u, torch.full((B,), 0.5, device=DEV), q=q, d_status=st,
                          max_path=8, **({"pos": step.tree.pos} if given else {}))
    layers.draft_accept(caches, state, step, v, d_status=st)
    keep = v.keep.tolist()
    others = [b for b in range(B) if b != bad]
    assert all(keep[b] > 1 for b in others) and int(st) & csa2.DEV_BAD_INDEX
    if given:
        assert keep[bad] == 0 and int(v.token[bad]) == -1 and v.path[bad].tolist() == [-1] * 8
    assert state.lens.tolist() == [n + (0 if b == bad else keep[b]) for b, n in enumerate(before)]
    assert v.delta.tolist() == [-sizes[b] if b == bad else keep[b] - sizes[b] for b in range(B)]
    held = [-(-n // page) for n in state.lens.tolist()]
    assert int(state.n_free) == 200 - sum(held) and int(state.n_free) <= n_free
    ids = [int(v) for b in range(B) for v in state.block_table[b, :held[b]]] + state.free_pages[:int(state.n_free)].tolist()
    assert sorted(ids) == list(range(200))
    for c, rows in zip(caches, old):
        for x, y in zip(raw(c), rows):
            assert np.array_equal(x[state.block_table[bad, :held[bad]].cpu().numpy()].reshape(-1, x.shape[2])[:before[bad]], y)


def test_a_request_that_ends_with_its_step():
    # the server gives a delta of its own: the request's rows all go, its path is moved or not
    page, H, d, B, g = 16, 4, 64, 2, torch.Generator(device=DEV).manual_seed(4)
    cache, state = paged.PagedCache.new(30, page, d), layers.PagedState(ints([0] * B), ints(np.full((B, 10), -1)), ints(range(30)), ints([30]))
    x = lambda delta: layers.PagedInput(torch.randn((sum(delta), H, d), generator=g, device=DEV).bfloat16(),  # noqa: E731
                                        torch.randn((sum(delta), d), generator=g, device=DEV).bfloat16(), ints(delta))
    layers.paged_layer(cache, state, x([40, 20]), 0, d)
    step = layers.draft_plan(page, state, x([4, 4]), ints([-1, 0, 1, 0] * 2), 4)
    v = draft.Verdict(ints([2, 2]), ints([[0, 3], [0, 3]]), ints([1, 1]), ints([-44, -2]))
    st = status()
    layers.draft_accept([cache], state, step, v, d_status=st)
    assert int(st) == 0 and state.lens.tolist() == [0, 22] and int(state.n_free) == 28 and v.delta.tolist() == [-44, -2]
