"""Drafted tokens and shared pages on the GPU against plain implementations in whole numbers and in 64 bits."""
import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_gb300 import csa2, draft, layers, paged
from test_gpu_paged import DEV, FMTS, I32, close, cos_sin, ints, random_cache, status, values64

pytestmark = pytest.mark.gpu


def random_tree(r, n, shape="tree"):
    """Parents of n nodes: a chain, a tree, several trees, or a star."""
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "star":
        return ([-1] + [0] * (n - 1))[:n]
    if shape == "forest":
        return [-1 if i == 0 or r.random() < 0.3 else int(r.integers(0, i)) for i in range(n)]
    return [-1 if i == 0 else int(r.integers(max(0, i - 6), i)) for i in range(n)]


def ways(parent):
    """Each node's way up to its root, itself first."""
    out = []
    for i, p in enumerate(parent):
        out.append([i] + (out[p] if 0 <= p < i else []))
    return out


# ------------------------------------------------------------------ positions and masks
def tree_ref(parent, lens, cu, words):
    T, B = len(parent), len(lens)
    pos, seen, st = np.full(T, -1, dtype=np.int64), np.zeros((T, words), dtype=np.uint32), 0
    held = [min(max(c, 0), T) for c in cu]
    if any(b < a for a, b in zip(held, held[1:])):
        return pos, seen, csa2.DEV_BAD_INDEX
    for b in range(B):
        c0, n = cu[b], cu[b + 1] - cu[b]
        if n <= 0:
            continue
        if c0 < 0 or c0 + n > T or n > 32 * words or lens[b] < n:
            st |= csa2.DEV_BAD_INDEX
            continue
        mine = [int(v) for v in parent[c0:c0 + n]]
        if any(not -1 <= p < i for i, p in enumerate(mine)):
            st |= csa2.DEV_BAD_INDEX
        for i, way in enumerate(ways(mine)):
            pos[c0 + i] = lens[b] - n + len(way) - 1
            for k in way:
                seen[c0 + i, k // 32] |= np.uint32(1 << (k % 32))
    return pos, seen, st


def run_tree_plan(parent, lens, cu, max_nodes):
    words = -(-max_nodes // 32)
    T = len(parent)
    out = draft.TreePlan(torch.full((T,), 7, dtype=I32, device=DEV), torch.full((T, words), 7, dtype=I32, device=DEV))
    st = status()
    draft.tree_plan(ints(parent), ints(lens), ints(cu), max_nodes, d_status=st, out=out)
    pos, seen, want = tree_ref(parent, lens, cu, words)
    assert out.pos.tolist() == pos.tolist()
    assert np.array_equal(out.seen.cpu().numpy().view(np.uint32), seen)
    assert int(st) == want
    return out


@pytest.mark.parametrize("shape", ["chain", "tree", "forest", "star"])
@pytest.mark.parametrize("sizes,max_nodes", [([1], 1), ([6], 32), ([32, 33, 1, 0, 64], 64), ([1, 0, 0, 5], 5), ([200, 31, 128], 200), ([1024, 1000], 1024),
                                             ([3] * 700, 3), ([0, 0], 4)])
def test_tree_plan(sizes, max_nodes, shape):
    r = np.random.default_rng(sum(sizes) + max_nodes)
    parent = [p for n in sizes for p in random_tree(r, n, shape)]
    run_tree_plan(parent, [n + int(r.integers(0, 5000)) for n in sizes], np.cumsum([0] + sizes).tolist(), max_nodes)


@pytest.mark.parametrize("parent,lens,cu,max_nodes", [
    ([-1, 0, 5, 1, -2, 4, 6], [9], [0, 7], 32),                            # parents that are no lower node
    ([-1, 0, 2**31 - 1, -2**31], [9], [0, 4], 4),
    ([-1, 0, 1, 2, -1, 0], [9, 9], [0, 4, 6], 3),                           # (the masks' width counts: up to 32 nodes)
    ([-1] * 40 + [0] * 3, [90, 90], [0, 40, 43], 32),                       # more nodes than bits
    ([-1, 0, 1, -1, 0], [2, 9], [0, 3, 5], 8),                              # fewer rows than nodes
    ([-1, 0, 1, -1, 0], [-5, 9], [0, 3, 5], 8),
    ([-1, 0, 1, -1, 0], [9, 9], [0, 3, 7], 8),                              # nodes past the tokens
    ([-1, 0, 1, -1, 0], [9, 9], [-2, 3, 5], 8),                             # and before them
    ([-1, 0, 1, -1, 0], [9, 9], [1, 3, 4], 8),                              # tokens of no request at both ends
    ([-1, 0, 1, -1, 0], [9, 9, 9], [0, 3, 1, 5], 8),                        # offsets that step down
    ([-1, 0, 1, -1, 0], [9, 9, 9], [-3, -7, 0, 5], 8),                      # ... outside the tokens: they do not
    ([-1, 0], [2**31 - 1], [0, 2], 8), ([-1, 0, 0], [], [0], 8)])
def test_tree_plan_edges(parent, lens, cu, max_nodes):
    run_tree_plan(parent, lens, cu, max_nodes)


# ------------------------------------------------------------------ attention
class TreeCase:
    def __init__(self, lens, sizes, H, d, dv, fmt, page, window=0, start=None, shape="tree", seed=0, pad=0, q_scale=1.0, max_nodes=None, mask=None):
        self.g = torch.Generator(device=DEV).manual_seed(seed + 100)
        r = np.random.default_rng(seed)
        self.lens, self.sizes, self.H, self.d, self.dv, self.window, self.start = lens, sizes, H, d, dv, window, start
        need = [-(-n // page) for n in lens]
        self.cache = random_cache(sum(need) + 3, page, d, fmt, seed)
        order = torch.randperm(sum(need) + 3, generator=self.g, device=DEV).tolist()
        self.table = np.full((len(lens), max(need + [0]) + 2), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        T = sum(sizes) + pad
        self.q = (torch.randn((T, H, d), generator=self.g, device=DEV) * q_scale).bfloat16()
        self.cu = np.cumsum([0] + sizes).tolist()
        self.parents = [random_tree(r, n, shape) for n in sizes]
        self.sm = 1.0 / math.sqrt(d)
        self.words = -(-(max_nodes or max(sizes + [1])) // 32)
        pos, seen, _ = tree_ref([p for q in self.parents for p in q] + [-1] * pad, lens, self.cu, self.words)
        if mask is not None:                                               # bits of the caller's own
            seen = mask(r, seen)
        self.pos, self.seen = pos, seen

    def run(self, st=None, stream=None, **k):
        opt = dict(kv_start=ints(self.start) if self.start is not None else None, pos=ints(self.pos))
        opt.update(k)
        return draft.tree_attn(self.q, self.cache, torch.from_numpy(self.table).to(DEV).to(I32), ints(self.lens), ints(self.cu),
                               torch.from_numpy(self.seen.view(np.int32)).to(DEV), d_v=self.dv, window=self.window, sm_scale=self.sm, d_status=st,
                               stream=stream, **opt)

    def visible(self, b):
        """bool [nodes, rows] of request b."""
        n, size, c0 = self.lens[b], self.sizes[b], self.cu[b]
        base, start = n - size, max(self.start[b], 0) if self.start is not None else 0
        see = np.zeros((size, n), dtype=bool)
        for i in range(size):
            low = max(start, int(self.pos[c0 + i]) + 1 - self.window) if self.window else start
            see[i, :base] = np.arange(base) >= low
            for k in range(size):
                at = int(self.pos[c0 + k]) if self.window else base + k
                see[i, base + k] = bool(self.seen[c0 + i, k // 32] >> np.uint32(k % 32) & 1) and at >= low
        return see

    def ref(self):
        """(out, lse, bound of out, bound of lse) in 64 bits."""
        page, T = self.cache.page, self.q.shape[0]
        out = torch.zeros((T, self.H, self.dv), dtype=torch.float64, device=DEV)
        lse = torch.full((T, self.H), -math.inf, dtype=torch.float64, device=DEV)
        ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
        for b, n in enumerate(self.lens):
            t0, t1 = self.cu[b], self.cu[b + 1]
            if t1 <= t0:
                continue
            pages = torch.from_numpy(self.table[b, :-(-n // page)]).to(DEV)
            good = ((pages >= 0) & (pages < self.cache.n_pages)).repeat_interleave(page)[:n]
            pages = pages.clamp(0, self.cache.n_pages - 1)
            k = values64(self.cache.codes[pages].flatten(0, 1)[:n],
                         self.cache.scales[pages].flatten(0, 1)[:n] if self.cache.scales is not None else None, self.cache.fmt)
            see = torch.from_numpy(self.visible(b)).to(DEV) & good
            bad = ~torch.isfinite(k).all(1)
            kz = torch.where(bad[:, None], 0.0, k)
            for a in range(t0, t1, 64):                                    # 64 nodes at a time
                z = min(a + 64, t1)
                s, q = see[a - t0:z - t0], self.q[a:z].double()
                l = (torch.einsum("thd,jd->thj", q, kz) * self.sm).masked_fill(~s[:, None], -math.inf)
                top = l.amax(-1)
                some = top > -math.inf
                w = torch.exp(l - torch.where(some, top, 0.0)[..., None])
                tot = w.sum(-1)
                w = w / torch.where(some, tot, 1.0)[..., None]
                nan = (s & bad).any(1)
                o = w @ kz[:, :self.dv]
                o[nan] = math.nan
                out[a:z] = o
                lse[a:z] = torch.where(some, top + torch.log(torch.where(some, tot, 1.0)), -math.inf)
                lse[a:z][nan] = math.nan
                # as in test_gpu_paged: float32 sums of d products, scaled and raised; weights and results
                # rounded to bf16 (2^-8 each: half a step)
                mag = torch.einsum("thd,jd->thj", q.abs(), kz.abs()).masked_fill(~s[:, None], 0.0).amax(-1) * self.sm
                dl = mag * self.d * 2.0 ** -23 + 2.0 ** -20 + torch.where(some, top.abs(), 0.0) * 2.0 ** -21
                ob[a:z] = o.abs() * 2.0 ** -8 + (w @ kz[:, :self.dv].abs()) * (2.0 ** -8 + 2 * dl[..., None] + n * 2.0 ** -23) * 1.01 + 1e-30
                lb[a:z] = dl * 1.01 + n * 2.0 ** -23 + 2.0 ** -20
        return out, lse, ob, lb


def check(case, st_want=0, **k):
    st = status()
    out, lse = case.run(st, **k)
    o, l, ob, lb = case.ref()
    n = case.cu[-1]
    close(out[:n], o[:n], ob[:n])
    close(lse[:n], l[:n], lb[:n])
    assert int(st) == st_want
    return out, lse


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,d,dv", [(64, 576, 512), (16, 128, 128), (1, 32, 8), (128, 512, 512), (5, 96, 40), (33, 288, 264)])
def test_tree_attn_formats_and_heads(fmt, H, d, dv):
    check(TreeCase([300, 1, 77], [9, 1, 40], H, d, dv, fmt, 16, seed=H + fmt))


@pytest.mark.parametrize("lens,sizes,page", [
    ([1], [1], 64), ([64], [64], 64), ([65], [64], 64), ([128], [1], 128), ([129], [2], 128), ([257, 256, 255], [3, 2, 1], 32), ([1000], [7], 1),
    ([513], [513], 16), ([5000, 3, 700], [6, 3, 128], 64), ([20000], [6], 64), ([130] * 40, [6] * 40, 64), ([7, 0, 9], [1, 0, 9], 8), ([4096], [200], 4096),
    ([1024], [1024], 64), ([140, 200, 260], [13, 72, 133], 16)])
@pytest.mark.parametrize("shape", ["chain", "tree"])
def test_tree_attn_lengths(lens, sizes, page, shape):
    check(TreeCase(lens, sizes, 64 if sum(sizes) < 300 else 16, 576, 512, paged.MXFP4, page, shape=shape, seed=lens[0]))


@pytest.mark.parametrize("window,start", [(1, None), (2, None), (5, None), (20, None), (128, None), (1000, None), (0, [3, 290, 0]), (7, [280, 1000, 199]),
                                          (0, [1000, 300, -5]), (2**31 - 1, None)])
@pytest.mark.parametrize("shape", ["chain", "tree", "forest"])
def test_tree_attn_windows(window, start, shape):
    # shorter than the trees are deep, and longer; rows that kv_start leaves out, the drafts' among them
    check(TreeCase([300, 310, 200], [40, 3, 70], 16, 128, 128, paged.NVFP4_E4M3_16, 16, window, start, shape, seed=window % 1000))


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("H", [1, 16, 64])
@pytest.mark.parametrize("kind", ["random", "none", "all", "holes"])
def test_tree_attn_masks_of_the_callers(kind, H, window):
    # any bits: some above a node's own place, some past the last node, none at all
    def mask(r, seen):
        if kind == "none":
            return np.zeros_like(seen)
        if kind == "all":
            return np.full_like(seen, 0xFFFFFFFF)
        m = r.integers(0, 2**32, seen.shape, dtype=np.uint32)
        if kind == "holes":
            m[r.random(len(m)) < 0.5] = 0
        return m
    c = TreeCase([50, 45, 290], [45, 45, 70], H, 128, 128, paged.MXFP4, 16, window, None, seed=H, max_nodes=96, mask=mask)
    out, lse = check(c)
    if kind == "none":                                                     # the second has no other rows
        assert bool((out[45:90] == 0).all()) and bool((lse[45:90] == -math.inf).all())


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("H,lens,sizes,max_nodes", [(64, [400], [300], 1024), (128, [350, 90], [300, 40], 320), (16, [260], [200], 192 + 8), (16, [260], [200], 256),
                                                    (1, [700], [640], 1024), (8, [130, 257], [130, 128], 130)])
@pytest.mark.parametrize("kind", ["tree", "holes"])
def test_tree_attn_wide_masks(kind, H, lens, sizes, max_nodes, window):
    # masks of many words, where a row tile's tokens are looked through for the nodes they see, and where not
    def mask(r, seen):
        return np.where(r.random(seen.shape) < 0.7, 0, r.integers(0, 2**32, seen.shape, dtype=np.uint32) & r.integers(0, 2**32, seen.shape, dtype=np.uint32)).astype(np.uint32)
    check(TreeCase(lens, sizes, H, 128, 128, paged.MXFP8, 32, window, None, seed=H + max_nodes, max_nodes=max_nodes, mask=mask if kind == "holes" else None))


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.BF16])
def test_tree_attn_strided_pages(fmt):
    c = TreeCase([300, 100], [25, 6], 64, 576, 512, fmt, 16, seed=14)
    want, n = c.run(), c.cache.n_pages
    codes = torch.zeros((n, 3, 16, c.cache.codes.shape[2]), device=DEV, dtype=c.cache.codes.dtype)
    codes[:, 2] = c.cache.codes
    if fmt == paged.BF16:
        c.cache = paged.PagedCache(codes[:, 2])
    else:
        scales = torch.full((n, 2, 16, c.cache.scales.shape[2]), 255, device=DEV, dtype=torch.uint8)
        scales[:, 1] = c.cache.scales
        c.cache = paged.PagedCache(codes[:, 2], scales[:, 1])
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tree_attn_of_a_chain_is_paged_attn():
    c = TreeCase([3000, 400], [6, 6], 64, 576, 512, paged.MXFP4, 64, shape="chain", seed=3)
    out, lse = c.run()
    o2, l2 = paged.paged_attn(c.q, c.cache, torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu), d_v=512, sm_scale=c.sm)
    _, _, ob, lb = c.ref()
    close(out, o2.double(), 2 * ob)
    close(lse, l2.double(), 2 * lb)


def test_tree_attn_large_logits():
    check(TreeCase([700, 300], [3, 20], 64, 576, 512, paged.MXFP4, 32, q_scale=30.0, seed=4))


@pytest.mark.parametrize("fmt", FMTS)
def test_tree_attn_not_finite_rows(fmt):
    # a drafted row that is not finite: the nodes below it become NaN and no others
    c = TreeCase([200, 150], [60, 60], 16, 128, 128, fmt, 16, seed=10)
    for b, j in ((0, 150), (1, 149), (0, 203)):                            # 203: past the rows held
        pg, off = int(c.table[b, j // 16]), j % 16
        if fmt == paged.BF16:
            c.cache.codes[pg, off, 5] = math.inf
        else:
            c.cache.scales[pg, off, 1] = 0x7F if fmt == paged.NVFP4_E4M3_16 else 255
    out, _ = check(c)
    bits = sum(int(v) >> 10 & 1 for v in c.seen[:60, 0]) + 1
    assert int(torch.isnan(out).any(-1).any(-1).sum()) == bits


def test_tree_attn_bad_pages():
    c = TreeCase([300, 400, 200], [14, 2, 30], 64, 576, 512, paged.MXFP4, 16, seed=7)
    c.table[0, 3], c.table[0, 18], c.table[1, 0], c.table[2, 1:] = -1, 2**31 - 1, c.cache.n_pages, -2**31
    check(c, csa2.DEV_BAD_INDEX)


def test_tree_attn_rows_past_the_table():
    c = TreeCase([300, 100], [40, 9], 16, 128, 128, paged.MXFP4, 16, seed=9)
    cut = c.table.copy()
    cut[0, 18:] = -1                                                       # what a table of 18 entries reaches
    c.table = cut
    want = check(c, csa2.DEV_BAD_INDEX)
    c.table, st = np.ascontiguousarray(cut[:, :18]), status()
    got = c.run(st)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(st) == csa2.DEV_BAD_INDEX


def test_tree_attn_requests_left_out():
    # more nodes than bits, fewer rows than nodes, nodes outside q: their rows stay as they were
    c = TreeCase([300, 300, 300, 300], [5, 40, 3, 6], 16, 128, 128, paged.MXFP4, 16, seed=12, pad=5)
    want = c.run()[0]
    out = torch.full((59, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((59, 16), 4.0, device=DEV)
    c.lens, c.seen, st = [300, 300, 2, 300], np.ascontiguousarray(c.seen[:, :1]), status()
    c.run(st, out=out, lse=lse)
    assert int(st) == csa2.DEV_BAD_INDEX
    assert torch.equal(out[:5], want[:5]) and torch.equal(out[48:54], want[48:54])
    assert bool((out[5:48] == 3.0).all()) and bool((lse[5:48] == 4.0).all()) and bool((out[54:] == 3.0).all())
    c.lens, c.cu = [300] * 4, [0, 5, 5, 53, 60]                            # the third too many nodes, the fourth past the end
    out.fill_(3.0), st.zero_()
    c.run(st, out=out)
    assert int(st) == csa2.DEV_BAD_INDEX and torch.equal(out[:5], want[:5]) and bool((out[5:] == 3.0).all())


@pytest.mark.parametrize("cu", [[0, 5, 0, 5], [0, 3, 1, 5], [5, 0, 5, 5]])
def test_tree_attn_offsets_that_step_down(cu):
    c = TreeCase([40, 37, 33], [5, 0, 0], 64, 128, 128, paged.MXFP4, 32, seed=21)
    c.cu, st = cu, status()
    out = torch.full((5, 64, 128), 3.0, device=DEV).bfloat16()
    c.run(st, out=out)
    assert int(st) == csa2.DEV_BAD_INDEX and bool((out == 3.0).all())


@pytest.mark.parametrize("pos", [-2**31, 2**31 - 1, -1])
def test_tree_attn_wild_positions(pos):
    # positions that no plan gives: nothing outside the tables is read, and rows are weighed as they say
    c = TreeCase([140, 90], [9, 3], 16, 128, 128, paged.MXFP4, 16, window=50, seed=22)
    c.pos[4] = pos
    check(c)


def test_tree_attn_same_twice_streams_and_graphs():
    cs = [TreeCase([6000, 500], [6, 30], 64, 576, 512, paged.MXFP4, 64, seed=s) for s in (17, 18)]
    want = [c.run() for c in cs]
    ws = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        b = cs[0].run(workspace=ws)
        assert torch.equal(b[0], want[0][0]) and torch.equal(b[1], want[0][1])
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(c.run())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # captured: positions, masks and attention, replayed with new lengths and trees
    c = cs[0]
    table, lens, cu = torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu)
    parent = ints([p for q in c.parents for p in q])
    out, lse, plan = torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), draft.tree_plan(parent, lens, cu, 30)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        draft.tree_plan(parent, lens, cu, 30, out=plan)
        draft.tree_attn(c.q, c.cache, table, lens, cu, plan.seen, plan.pos, d_v=512, sm_scale=c.sm, out=out, lse=lse, workspace=ws)
    r = np.random.default_rng(5)
    for new_lens in ([6000, 500], [40, 480], [5990, 31]):
        c.lens, c.parents = new_lens, [random_tree(r, n) for n in c.sizes]
        lens.copy_(ints(new_lens)), parent.copy_(ints([p for q in c.parents for p in q]))
        g.replay()
        c.pos, c.seen, _ = tree_ref([p for q in c.parents for p in q], new_lens, c.cu, 1)
        o, l, ob, lb = c.ref()
        close(out, o, ob)
        close(lse, l, lb)


def test_tree_attn_given_stream():
    c = TreeCase([3000], [25], 64, 576, 512, paged.MXFP4, 64, seed=19)
    want, s = c.run(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ verification
ONE = 1 << 40
F = np.float32


def whole(w):
    """Weights as whole numbers of 2^-40."""
    return np.rint(np.minimum(w, F(1.0)).astype(np.float64) * ONE).astype(np.int64)


def clean(v, st):
    ok = (v >= 0) & np.isfinite(v)
    if not ok.all():
        st[0] |= csa2.DEV_NONFINITE
    return np.where(ok, v, F(0.0)).astype(F)


def verify_ref(p, q, token, parent, cu, u, r, max_path):
    """Request by request, child by child; float32 operations one by one, sums in whole numbers."""
    T, V = p.shape
    B, st = len(r), [0]
    keep, path, nxt, delta = [], np.full((B, max_path), -1, dtype=np.int64), [], []
    for b in range(B):
        c0, n = cu[b], cu[b + 1] - cu[b]
        if n <= 0 or c0 < 0 or c0 + n > T or n > 1024:
            st[0] |= csa2.DEV_BAD_INDEX if n > 0 else 0
            keep.append(0), nxt.append(-1), delta.append(0)
            continue
        kids = [[] for _ in range(n)]
        for i in range(1, n):
            up = int(parent[c0 + i])
            if -1 <= up < i:
                if up >= 0:
                    kids[up].append(i)
            else:
                st[0] |= csa2.DEV_BAD_INDEX
        at, kept = 0, [0]
        while True:
            c, m, gone, weights, down = F(0.0), F(1.0), set(), None, None
            for i in kids[at] if len(kept) < max_path else []:
                x = int(token[c0 + i])
                if not 0 <= x < V:
                    st[0] |= csa2.DEV_BAD_INDEX
                    continue
                px = clean(p[c0 + at, x:x + 1], st)[0]
                if q is not None:
                    qx = clean(q[c0 + at, x:x + 1], st)[0]
                    if u[c0 + i] * qx * m < max(px - c * qx, F(0.0)):
                        down = i
                        break
                    c = F(c + m)
                    row, other = clean(p[c0 + at], st), clean(q[c0 + at], st)
                    weights = whole(np.maximum(row - c * other, F(0.0)))
                    m = F(int(weights.sum())) * F(2.0 ** -40)
                else:
                    if x in gone:
                        px = F(0.0)
                    if u[c0 + i] * m < px:
                        down = i
                        break
                    m = max(F(m - px), F(0.0))
                    gone.add(x)
            if down is None:
                break
            at = down
            kept.append(at)
        if weights is None:
            weights = whole(clean(p[c0 + at], st))
            weights[list(gone)] = 0
        if weights.sum() == 0:
            weights = whole(clean(p[c0 + at], st))
        total = int(weights.sum())
        mm = F(r[b]) * F(2.0 ** 24)
        mm = 0 if np.isnan(mm) else int(min(max(math.floor(mm) if np.isfinite(mm) else (2**24 if mm > 0 else 0), 0), 2**24 - 1))
        if total == 0:
            st[0] |= draft.DEV_NO_TOKEN
            nxt.append(-1)
        else:
            nxt.append(int(np.searchsorted(np.cumsum(weights), total * mm >> 24, side="right")))
        keep.append(len(kept)), delta.append(len(kept) - n)
        path[b, :len(kept)] = kept
    return keep, path.tolist(), nxt, delta, st[0]


class VerifyCase:
    def __init__(self, sizes, V, dtype=torch.float32, drawn=True, shape="tree", near=0.7, seed=0, pad=0, sharp=2.0):
        r = np.random.default_rng(seed)
        self.cu = np.cumsum([0] + sizes).tolist()
        T = sum(sizes) + pad
        z = r.standard_normal((T, V)) * sharp
        y = z + r.standard_normal((T, V)) * near
        soft = lambda a: np.exp(a - a.max(1, keepdims=True)) / np.exp(a - a.max(1, keepdims=True)).sum(1, keepdims=True)  # noqa: E731
        self.p = torch.from_numpy(soft(z)).to(dtype)
        self.q = torch.from_numpy(soft(y)).to(dtype) if drawn else None
        self.parent = np.array([p for n in sizes for p in random_tree(r, n, shape)] + [-1] * pad, dtype=np.int64)
        self.token = np.zeros(T, dtype=np.int64)
        for b, n in enumerate(sizes):
            for i in range(1, n):
                up = self.parent[self.cu[b] + i]
                noise = r.gumbel(size=V)
                self.token[self.cu[b] + i] = int(np.argmax(y[self.cu[b] + max(up, 0)] + noise))
        self.u, self.r = r.random(T).astype(F), r.random(len(sizes)).astype(F)

    def run(self, max_path=None, st=None, stream=None, p=None, q=None, out=None):
        p = self.p.to(DEV) if p is None else p
        q = (self.q.to(DEV) if self.q is not None else None) if q is None else q
        return draft.tree_verify(p, ints(self.token), ints(self.parent), ints(self.cu), torch.from_numpy(self.u).to(DEV),
                                 torch.from_numpy(self.r).to(DEV), q=q, max_path=max_path, d_status=st, stream=stream, out=out)

    def check(self, max_path=None, **k):
        st = status()
        v = self.run(max_path, st, **k)
        L = v.path.shape[1]
        want = verify_ref(self.p.float().numpy(), self.q.float().numpy() if self.q is not None else None, self.token, self.parent, self.cu, self.u,
                          self.r, L)
        assert v.keep.tolist() == want[0] and v.path.tolist() == want[1]
        assert v.token.tolist() == want[2] and v.delta.tolist() == want[3]
        assert int(st) == want[4]
        return v


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("sizes,V", [([6], 32000), ([1], 7), ([3, 1, 9, 0, 33], 1), ([5, 5, 5], 2), ([40, 12, 64, 2], 31), ([9] * 20, 1000), ([16, 7, 1], 32003),
                                     ([6, 9], 131072), ([5], 1 << 18), ([4] * 200, 515), ([300, 1024], 66), ([3] * 700, 64)])
def test_verify(sizes, V, drawn, dtype):
    for shape in ("tree", "star"):
        VerifyCase(sizes, V, dtype, drawn, shape, seed=V + len(sizes)).check()


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_finds_every_outcome(drawn):
    # near and far drafts: nothing kept, all kept, siblings tried one after another
    seen = set()
    for near, seed in ((0.0, 1), (0.5, 2), (6.0, 3)):
        v = VerifyCase([8] * 60, 300, drawn=drawn, shape="tree", near=near, seed=seed).check()
        seen |= {int(k) for k in v.keep}
    assert ({1, 2, 3, 4} if drawn else {1, 2}) <= seen                     # (certain drafts are a target's token less often)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,row,first", [(1000, 1003, 0), (1000, 1024, 1), (1001, 1008, 8), (4099, 4104, 16), (33, 40, 0)])
def test_verify_strided_rows(V, row, first, dtype):
    # rows that begin on any value, and rows of a padded vocabulary, what is behind them not read
    c = VerifyCase([6, 9, 2], V, dtype, seed=V)
    wide = [torch.full((17, row + first), math.nan, dtype=dtype, device=DEV) for _ in range(2)]
    views = [w[:, first:first + V] for w in wide]
    views[0].copy_(c.p), views[1].copy_(c.q)
    c.check(p=views[0], q=views[1])
    c.check(p=views[0])


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_numbers_at_the_ends(drawn):
    c = VerifyCase([7] * 12, 200, drawn=drawn, seed=30, near=1.5)
    for u, r in ((0.0, 0.0), (1.0, 1.0), (1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24), (math.nan, math.nan), (-1.0, -3.0), (7.0, math.inf)):
        c.u[:], c.r[:] = u, r
        v = c.check()
        if u == 1.0 - 2.0 ** -24 and drawn:
            c.q = c.p                                                      # equal distributions: nothing is turned down
            assert all(k > 1 for k in c.check().keep.tolist())
            c = VerifyCase([7] * 12, 200, drawn=drawn, seed=31, near=1.5)
        assert bool((v.token >= 0).all())


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_certain_targets(drawn):
    # the target's distribution is one token: drafts stay while they are that token, and it follows
    c = VerifyCase([6] * 20, 50, drawn=drawn, shape="chain", seed=32, sharp=0.5)
    best = c.p.argmax(1)
    c.p = torch.nn.functional.one_hot(best, 50).float()
    for b in range(20):
        for i in range(1, 6):
            if (b + i) % 3:
                c.token[6 * b + i] = int(best[6 * b + i - 1])
    v = c.check()
    for b in range(20):
        k = 1
        while k < 6 and c.token[6 * b + k] == int(best[6 * b + k - 1]):
            k += 1
        assert int(v.keep[b]) == k and int(v.token[b]) == int(best[6 * b + k - 1])


def test_verify_weights_that_are_none():
    # nothing left, nothing at all, values below 0 and not finite, tokens outside the vocabulary
    c = VerifyCase([4, 4, 4, 4, 4, 4], 37, seed=33, shape="star")
    c.p[0], c.q[0] = 0.0, 1.0 / 37                                         # no weight: no token
    c.p[4, :], c.q[4, :] = 0.0, 0.0
    c.p[4, 5], c.q[4, 5], c.q[4, 6], c.token[5:8] = 0.5, 1.0, 0.5, 6         # q covers p: p itself is drawn from
    c.p[8, 3], c.p[8, 4], c.p[8, 5], c.q[8, 7] = math.nan, -1.0, math.inf, math.inf
    c.token[9], c.token[10], c.token[11] = 3, 5, 7
    c.token[13], c.token[14], c.token[15] = -1, 37, 2**31 - 1
    c.p[16] = 5.0                                                          # more than 1: held
    c.p[20], c.q[20] = 1e-20, 1e-30                                        # below the weights' step: drafts stay all the same
    v = c.check()
    assert v.token[0] == -1 and v.token[1] == 5 and v.keep[5] == 2
    c.q = None
    c.check()


def test_verify_paths_and_requests():
    # paths cut off, requests without nodes, out of range, parents that are none
    c = VerifyCase([9, 0, 7, 5], 60, near=0.1, seed=34, shape="chain")
    for max_path in (1, 2, 3, 9, 50):
        c.check(max_path)
    c.parent[3], c.parent[12] = 5, -7
    c.check()
    c.cu = [0, 9, 9, 16, 40]
    c.check(9)
    c.cu = [-1, 9, 3, 16, 21]
    c.check(9)


def test_verify_is_deterministic_in_streams_and_graphs():
    cs = [VerifyCase([6, 16, 9], 50000, seed=s, near=1.5) for s in (35, 36)]
    want = [c.check(16) for c in cs]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(c.run(16))
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(getattr(a, f), getattr(b, f)) for f in ("keep", "path", "token", "delta"))  # noqa: E731
    assert all(same(a, b) for a, b in zip(got, want))
    c = cs[0]
    p, q, u, r = c.p.to(DEV), c.q.to(DEV), torch.from_numpy(c.u).to(DEV), torch.from_numpy(c.r).to(DEV)
    token, parent, cu, out = ints(c.token), ints(c.parent), ints(c.cu), c.run(16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        draft.tree_verify(p, token, parent, cu, u, r, q=q, max_path=16, out=out)
    for c in cs:
        p.copy_(c.p), q.copy_(c.q), u.copy_(torch.from_numpy(c.u)), r.copy_(torch.from_numpy(c.r)), token.copy_(ints(c.token)), parent.copy_(ints(c.parent))
        g.replay()
        assert same(out, want[cs.index(c)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cs[1].run(16, stream=s)
    s.synchronize()
    assert same(got, want[1])


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_gives_the_targets_distribution(drawn):
    # one tree of two levels, 16,384 times with other drafts and numbers: the first token behind the root is
    # distributed as the target's row, kept or not.  A share of N draws is off by more than 6 sqrt(p (1 - p) / N)
    # once in 5e8
    V, N, r = 8, 16384, np.random.default_rng(37)
    p0, q0 = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    parent = [-1, 0, 0, 0]
    T = 4 * N
    p = torch.from_numpy(np.tile(np.stack([p0, r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))]), (N, 1)).astype(F))
    q = torch.from_numpy(np.tile(q0, (T, 1)).astype(F))
    token = r.choice(V, size=T, p=q0) if drawn else np.tile([0, 1, 5, 3], N)
    v = draft.tree_verify(p.to(DEV), ints(token), ints(parent * N), ints(range(0, T + 1, 4)), torch.from_numpy(r.random(T).astype(F)).to(DEV),
                          torch.from_numpy(r.random(N).astype(F)).to(DEV), q=q.to(DEV) if drawn else None, max_path=4)
    keep, path, nxt = v.keep.cpu().numpy(), v.path.cpu().numpy(), v.token.cpu().numpy()
    first = np.where(keep > 1, token[4 * np.arange(N) + np.maximum(path[:, 1], 0)], nxt)
    share = np.bincount(first, minlength=V) / N
    assert (np.abs(share - p0) <= 6 * np.sqrt(p0 * (1 - p0) / N) + 1e-6).all()
    assert 0.1 < (keep > 1).mean() < 0.99


# ------------------------------------------------------------------ pages
def bytes_cache(n_pages, page, d, fmt, seed, strided=False):
    """A cache of any bytes; strided: pages between another layer's, scales on odd addresses where they may."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = paged.PagedCache.new(1, 1, d, fmt, device="cpu")
    layers_ = 2 if strided else 1
    width = shape.codes.shape[2] * (2 if fmt == paged.BF16 else 1)
    codes = torch.randint(0, 256, (n_pages, layers_, page, width), generator=g, device=DEV, dtype=torch.uint8)
    if fmt == paged.BF16:
        return paged.PagedCache(codes.view(torch.bfloat16)[:, -1])
    s = shape.scales.shape[2]
    odd = 2 if fmt == paged.NVFP4_E4M3_16 else 1
    scales = torch.randint(0, 256, (n_pages * layers_ * page * s + odd,), generator=g, device=DEV, dtype=torch.uint8)
    scales = scales[odd if strided else 0:][:n_pages * layers_ * page * s].view(n_pages, layers_, page, s)
    return paged.PagedCache(codes[:, -1], scales[:, -1])


def raw(cache):
    """Bytes of codes and scales, as [n_pages, page, bytes] on the host."""
    codes = cache.codes.contiguous().view(torch.uint8).view(cache.n_pages, cache.page, -1)
    return [t.cpu().numpy().copy() for t in (codes, cache.scales) if t is not None]


def table_of(r, lens, page, n_pages, width):
    need = [-(-max(n, 0) // page) for n in lens]
    ids = r.permutation(n_pages)
    table = np.full((len(lens), width), -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:].tolist()


def compact_ref(data, table, lens, cu, path, keep, page, n_pages):
    st = 0
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        base, way = lens[b] - n, [int(v) for v in path[b][:max(keep[b], 0)]]
        if keep[b] == 0:
            continue
        if keep[b] < 0 or keep[b] > path.shape[1] or n < 0 or base < 0 or any(y <= x for x, y in zip([-1] + way, way)) or way[-1] >= n:
            st |= csa2.DEV_BAD_INDEX
            continue
        slots = []
        for i, at in enumerate(way):
            ends = []
            for row in (base + at, base + i):
                j = row // page
                pg = int(table[b, j]) if j < table.shape[1] else -1
                ends.append((pg, row % page) if 0 <= pg < n_pages else None)
            if at != i:
                if None in ends:
                    st |= csa2.DEV_BAD_INDEX
                else:
                    slots.append(ends)
        for t in data:
            rows = [t[a].copy() for a, _ in slots]
            for v, (_, z) in zip(rows, slots):
                t[z] = v
    return st


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,page,most,d,strided", [(1, 64, 6, 576, False), (9, 16, 40, 128, True), (40, 1, 25, 32, False), (7, 128, 300, 1024, True), (300, 4, 9, 64, True)])
def test_compact(fmt, B, page, most, d, strided):
    r = np.random.default_rng(B + fmt)
    sizes = [int(r.integers(0, most + 1)) if b else most for b in range(B)]
    lens = [n + int(r.integers(0, 3 * page + 5)) for n in sizes]
    n_pages = sum(-(-n // page) for n in lens) + 3
    table, _ = table_of(r, lens, page, n_pages, max(-(-n // page) for n in lens) + 1)
    keep = [int(r.integers(0, min(n, 30) + 1)) for n in sizes]
    path = np.full((B, 30), -1)
    for b, (n, k) in enumerate(zip(sizes, keep)):
        path[b, :k] = np.sort(r.choice(n, k, replace=False)) if k else []
    cu = np.cumsum([0] + sizes).tolist()
    caches = [bytes_cache(n_pages, page, d, fmt, seed, strided) for seed in (1, 2, 3)]
    before = [raw(c) for c in caches]
    st = status()
    draft.paged_compact(caches, ints(table), ints(lens), ints(cu), ints(path), ints(keep), d_status=st)
    for c, want in zip(caches, before):
        assert compact_ref(want, table, lens, cu, path, keep, page, n_pages) == 0
        assert all(np.array_equal(a, b) for a, b in zip(raw(c), want))
    assert int(st) == 0


def test_compact_refuses_and_passes_over():
    page, n_pages = 8, 40
    r = np.random.default_rng(4)
    lens, sizes = [30, 30, 30, 30, 30, 30, 3, 30, 30], [20, 20, 20, 20, 20, 20, 5, 20, 20]
    table, _ = table_of(r, lens, page, n_pages, 4)
    path = np.tile(np.array([1, 3, 4, 9, 19]), (9, 1))
    path[0, 2], path[1, 4], path[2, 0], path[3, 3] = 3, 20, -1, 2            # not rising, past the nodes, below 0, falling
    keep = [5, 5, 5, 5, 6, -1, 2, 5, 4]
    table[7, 1], table[8, 2] = -1, n_pages                                   # rows that have no page at either end
    cu = np.cumsum([0] + sizes).tolist()
    cache = bytes_cache(n_pages, page, 64, paged.MXFP4, 5)
    want, st = raw(cache), status()
    draft.paged_compact([cache], ints(table), ints(lens), ints(cu), ints(path), ints(keep), d_status=st)
    assert compact_ref(want, table, lens, cu, path, keep, page, n_pages) == int(st) == csa2.DEV_BAD_INDEX
    assert all(np.array_equal(a, b) for a, b in zip(raw(cache), want))


def test_compact_many_caches():
    # more than one call holds, of unlike widths and formats
    page, r = 16, np.random.default_rng(6)
    table, _ = table_of(r, [50, 40], page, 12, 5)
    caches = [bytes_cache(12, page, (64, 96, 576)[i % 3], FMTS[i % 4], i, i % 2 == 1) for i in range(35)]
    before = [raw(c) for c in caches]
    args = (table, [50, 40], [0, 9, 21], np.array([[0, 4, 8, -1], [0, 1, 5, 11]]), [3, 4])
    draft.paged_compact(caches, *(ints(a) for a in args))
    for c, want in zip(caches, before):
        compact_ref(want, *args, page, 12)
        assert all(np.array_equal(a, b) for a, b in zip(raw(c), want))


class Pages:
    """Requests, tables, counts and the free list beside lists that say what they should be."""

    def __init__(self, B, W, n_pages, page):
        self.B, self.W, self.n_pages, self.page = B, W, n_pages, page
        self.lens, self.table = [0] * B, [[-1] * W for _ in range(B)]
        self.shares, self.free = [0] * n_pages, list(range(n_pages))
        self.t_lens, self.t_table, self.t_shares = ints(self.lens), ints(self.table), ints(self.shares)
        self.t_free, self.t_n = ints(self.free), ints([n_pages])

    def args(self):
        return self.t_lens, self.t_table, self.t_shares, self.t_free, self.t_n, self.page

    def grow(self, delta):
        paged.page_plan(self.t_lens, ints(delta), self.t_table, self.t_free, self.t_n, self.page, 0, in_place=True)
        for b, d in enumerate(delta):
            had, has = -(-self.lens[b] // self.page), -(-(self.lens[b] + d) // self.page)
            self.free += self.table[b][has:had]
        for b, d in enumerate(delta):
            had, has = -(-self.lens[b] // self.page), -(-(self.lens[b] + d) // self.page)
            for j in range(had, has):
                self.table[b][j] = self.free.pop()
            self.lens[b] += d

    def fork(self, source):
        want, st = [], 0
        n_free = len(self.free)
        new, taken = {}, 0
        for b, a in enumerate(source):
            if a < 0:
                want.append((-1, -1, 0))
                continue
            if a >= self.B or a == b or self.lens[b] > 0 or source[a] >= 0:
                want.append((-1, draft.REFUSED, 0))
                st |= csa2.DEV_BAD_INDEX
                continue
            n = self.lens[a]
            full, part = n // self.page, n % self.page
            last = self.table[a][full] if part else -1
            if part and 0 <= last < self.n_pages:
                taken += 1
                if taken > n_free:
                    want.append((-1, draft.REFUSED, 0))
                    st |= paged.DEV_NO_PAGES
                    continue
                want.append((last, self.free.pop(), part))
                new[b] = (a, full, want[-1][1])
            else:
                want.append((-1, -1, 0))
                new[b] = (a, full, last)
        for b, (a, full, last) in new.items():
            for j in range(full):
                self.table[b][j] = self.table[a][j]
                if 0 <= self.table[a][j] < self.n_pages:
                    self.shares[self.table[a][j]] += 1
            if self.lens[a] % self.page:
                self.table[b][full] = last
            self.lens[b] = self.lens[a]
        s = status()
        f = draft.page_fork(ints(source), *self.args(), d_status=s)
        assert list(zip(f.src.tolist(), f.dst.tolist(), f.rows.tolist())) == want and int(s) == st
        self.same()
        return f

    def end(self, ends):
        gone = []
        for b, e in enumerate(ends):
            if e:
                for j in range(-(-self.lens[b] // self.page)):
                    if 0 <= self.table[b][j] < self.n_pages:
                        self.shares[self.table[b][j]] -= 1
                self.lens[b] = 0
        for i in range(self.n_pages):
            if self.shares[i] < 0:
                gone.append(i)
                self.shares[i] = 0
        self.free += gone
        s = status()
        draft.page_free(ints(ends), *self.args(), d_status=s)
        assert int(s) == 0
        self.same()

    def same(self):
        n = len(self.free)
        assert self.t_lens.tolist() == self.lens and self.t_table.tolist() == self.table
        assert self.t_shares.tolist() == self.shares
        assert int(self.t_n) == n and self.t_free.tolist()[:n] == self.free
        # every page is free or held, as often as it is counted
        held = np.zeros(self.n_pages, dtype=int)
        for b in range(self.B):
            for j in range(-(-self.lens[b] // self.page)):
                if 0 <= self.table[b][j] < self.n_pages:
                    held[self.table[b][j]] += 1
        free = np.zeros(self.n_pages, dtype=int)
        free[self.free] += 1
        assert ((held == 0) == (free == 1)).all() and free.max(initial=0) <= 1 and (held[held > 0] - 1 == np.array(self.shares)[held > 0]).all()


@pytest.mark.parametrize("B,W,n_pages,page,most,seed", [(2, 4, 8, 16, 40, 0), (12, 30, 400, 4, 60, 1), (40, 9, 300, 1, 9, 2), (700, 6, 9000, 8, 30, 3),
                                                        (6, 3000, 12000, 2, 5000, 4), (30, 40, 100000, 64, 2000, 5)])
def test_forks_and_ends(B, W, n_pages, page, most, seed):
    # prompts grow, are forked, grow on, and end in any order; forks of forks
    r, P = np.random.default_rng(seed), Pages(B, W, n_pages, page)
    for step in range(8):
        room = [W * page - n for n in P.lens]
        grow = [int(min(r.integers(0, most + 1), m)) if n or b < max(1, B // 4) else 0 for b, (n, m) in enumerate(zip(P.lens, room))]
        while sum(-(-(n + g) // page) - -(-n // page) for n, g in zip(P.lens, grow)) > len(P.free):
            grow = [g // 2 for g in grow]
        P.grow(grow)
        P.same()
        held = [b for b in range(B) if P.lens[b] > 0]
        source = [-1] * B
        for b in range(B):
            if P.lens[b] == 0 and held and r.random() < 0.6:
                source[b] = int(r.choice(held))
        P.fork(source)
        P.end([int(r.random() < 0.3) for _ in range(B)])
    P.end([1] * B)
    assert sorted(P.free) == list(range(n_pages))


@pytest.mark.parametrize("W", [3, 33, 70])
@pytest.mark.parametrize("order", ["one after another", "in turn", "with gaps", "one alone"])
def test_forks_beside_one_another(W, order):
    # neighbours that hold the same pages: runs of every length, over and within groups of requests, with
    # requests between that are refused, end earlier, or hold pages of their own
    page, P = 2, Pages(23, W, 30 * W, 2)
    lens = [min(2 * W - 1, 5), 2 * W - 1, 2 * W - 2]
    P.grow(lens + [0] * 20)
    source = [-1] * 3 + {"one after another": [0] * 7 + [1] * 9 + [2] * 4, "in turn": [i % 3 for i in range(20)],
                         "with gaps": [1, 1, -1, 1, 1, 1, 50, 1, 0, 1, 2, 2, 4, 2, -1, -1, 2, 2, 2, 2], "one alone": [-1] * 19 + [1]}[order]
    P.fork(source)
    P.grow([0 if n == 0 or n == 2 * W else 1 for n in P.lens])
    P.same()
    P.end([int(b % 5 == 4) for b in range(23)])
    P.end([int(b < 9) for b in range(23)])
    P.end([1] * 23)
    assert sorted(P.free) == list(range(30 * W))


def test_fork_refusals():
    P = Pages(7, 4, 12, 4)
    P.grow([9, 0, 0, 0, 0, 6, 0])
    #   own source, holds rows, forked source, out of range, and two that are fine
    P.fork([-1, 1, 0, 2, 7, 0, 5])
    P.fork([-1, 2**31 - 1, -1, -1, -5, -1, -1])
    P = Pages(6, 4, 5, 4)                                                   # three pages held, two free: the third fork starves,
    P.grow([9, 0, 0, 0, 0, 0])                                               # a fork of full pages does not
    P.fork([-1, 0, 0, 0, -1, -1])
    P.end([1, 0, 0, 0, 0, 0])
    P.grow([0, -1, 0, 0, 0, 0])
    P.fork([-1, -1, -1, 1, 1, 1])
    P.end([1] * 6)


def test_fork_tables_with_holes():
    # pages dropped in front, an id that is none, a last page that is none, more rows than the table reaches
    page, W = 4, 4
    lens, table = [14, 0, 0, 14, 0, 40, 0], [[-1, 3, 99, 5], [-7] * W, [-7] * W, [6, 7, 8, -1], [-7] * W, [9, 10, 11, 12], [-7] * W]
    t = [ints(v) for v in (lens, table, [0] * 20, list(range(13, 20)) + [-1] * 13, [7])]
    st = status()
    f = draft.page_fork(ints([-1, 0, -1, -1, 3, -1, 5]), *t, page, d_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX | paged.DEV_TABLE_FULL
    assert list(zip(f.src.tolist(), f.dst.tolist(), f.rows.tolist())) == [(-1, -1, 0), (5, 19, 2), (-1, -1, 0), (-1, -1, 0), (-1, -1, 0), (-1, -1, 0),
                                                                           (-1, draft.REFUSED, 0)]
    assert t[1].tolist() == [table[0], [-1, 3, 99, 19], table[2], table[3], [6, 7, 8, -1], table[5], table[6]]
    assert t[0].tolist() == [14, 14, 0, 14, 14, 40, 0] and int(t[4]) == 6
    assert [i for i, v in enumerate(t[2].tolist()) if v] == [3, 6, 7, 8]
    st.zero_()
    draft.page_free(ints([1, 1, 0, 1, 1, 1, 0]), *t, page, d_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX and t[0].tolist() == [0] * 7 and t[2].tolist() == [0] * 20
    assert int(t[4]) == 6 + 10 and t[3].tolist()[:16] == list(range(13, 19)) + [3, 5, 6, 7, 8, 9, 10, 11, 12, 19]


def test_free_list_without_room():
    t = [ints(v) for v in ([8, 4], [[0, 1], [2, -1]], [0] * 4, [3, -1], [1])]
    st = status()
    draft.page_free(ints([1, 1]), *t, 4, d_status=st)
    assert int(st) == paged.DEV_TABLE_FULL and int(t[4]) == 2 and t[3].tolist() == [3, 0] and t[2].tolist() == [0] * 4
    st.zero_()
    draft.page_free(ints([1, 1]), *t, 4, d_status=st)                       # ended already: nothing
    assert int(st) == 0 and int(t[4]) == 2


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page,d,strided", [(64, 576, False), (16, 128, True), (1, 32, True), (4096, 64, False), (8, 96, True)])
def test_copy(fmt, page, d, strided):
    r = np.random.default_rng(page)
    caches = [bytes_cache(23, page, d, fmt, s, strided) for s in (1, 2)]
    before = [raw(c) for c in caches]
    ids = r.permutation(23)
    src, dst = [int(v) for v in ids[:9]], [int(v) for v in ids[9:18]]
    src[4], dst[6], src[7] = -1, -2, dst[7]                                  # skipped; a page onto itself
    rows = [int(v) for v in r.integers(0, page + 1, 9)]
    rows[0], rows[1], rows[2] = -3, page + 5, page
    for given in (rows, None):
        st = status()
        draft.page_copy(caches, ints(src), ints(dst), ints(given) if given else None, d_status=st)
        for c, want in zip(caches, before):
            for a, z, n in zip(src, dst, given or [page] * 9):
                if a >= 0 and z >= 0:
                    for t in want:
                        t[z, :min(max(n, 0), page)] = t[a, :min(max(n, 0), page)]
            assert all(np.array_equal(x, y) for x, y in zip(raw(c), want))
        assert int(st) == 0
    small = bytes_cache(20, page, d, fmt, 3, strided)                        # a cache with fewer pages: flagged and skipped there
    want, st = raw(small), status()
    draft.page_copy([small], ints([20, 3, 2**31 - 1]), ints([1, 22, 2]), d_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX and all(np.array_equal(x, y) for x, y in zip(raw(small), want))


def test_pages_captured():
    # fork, copy and end in one graph, replayed over other requests
    P, page = Pages(6, 20, 100, 8), 8
    P.grow([50, 9, 0, 0, 0, 0])
    cache = bytes_cache(100, page, 64, paged.MXFP8, 1)
    source, ends = ints([-1] * 6), ints([0] * 6)
    f = draft.page_fork(source, *P.args())
    draft.page_copy([cache], f.src, f.dst, f.rows), draft.page_free(ends, *P.args())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        draft.page_fork(source, *P.args(), out=f)
        draft.page_copy([cache], f.src, f.dst, f.rows)
        draft.page_free(ends, *P.args())
    for s, e in (([-1, -1, 0, 0, 1, -1], [0, 0, 1, 0, 0, 0]), ([-1, -1, 1, -1, -1, 3], [1, 0, 0, 0, 1, 0]), ([-1] * 6, [1] * 6)):
        source.copy_(ints(s)), ends.copy_(ints(e))
        want = raw(cache)
        g.replay()
        for a, z, n in zip(f.src.tolist(), f.dst.tolist(), f.rows.tolist()):
            if a >= 0:
                for t in want:
                    t[z, :n] = t[a, :n]
        assert all(np.array_equal(x, y) for x, y in zip(raw(cache), want))
        lens = [P.lens[a] if a >= 0 else n for a, n in zip(s, P.lens)]
        P.lens = [0 if x else n for x, n in zip(e, lens)]
        assert P.t_lens.tolist() == P.lens
    assert sorted(P.t_free.tolist()) == list(range(100)) and int(P.t_n) == 100 and P.t_shares.tolist() == [0] * 100


def test_many_requests():
    # as many as a call takes: offsets, scans and tiles of 1,024 requests
    B, page, W = paged.MAX_BATCH, 4, 3
    r, n_pages = np.random.default_rng(8), 40000
    P = Pages(B, W, n_pages, page)
    P.grow([int(v) if b % 5 == 0 else 0 for b, v in enumerate(r.integers(1, W * page, B))])
    P.fork([-1 if b % 5 == 0 else int(r.integers(0, B // 5)) * 5 if r.random() < 0.9 else int(r.integers(0, B)) for b in range(B)])
    P.end([int(v) for v in r.random(B) < 0.5])
    P.end([1] * B)
    sizes = [int(v) for v in r.integers(0, 3, B)]
    parent = [p for n in sizes for p in random_tree(r, n)]
    run_tree_plan(parent, [n + int(v) for n, v in zip(sizes, r.integers(0, 9, B))], np.cumsum([0] + sizes).tolist(), 2)
    VerifyCase(sizes, 5, seed=9, near=1.0).check(3)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,window", [(paged.MXFP4, 0), (paged.NVFP4_E4M3_16, 40), (paged.MXFP8, 0), (paged.BF16, 9)])
def test_steps_of_a_server_with_drafts(fmt, window):
    """Two layers decode with trees of drafts: after each step the caches and the outputs of the kept nodes are those of
    the same tokens decoded one after another."""
    H, d, dv, rope, page, W, B, V = 16, 128, 128, 32, 16, 20, 3, 97
    r, g = np.random.default_rng(fmt), torch.Generator(device=DEV).manual_seed(fmt)
    cs = cos_sin(400, rope)
    rows = [torch.randn((V, d), generator=g, device=DEV).bfloat16() for _ in range(2)]       # each layer's row and query of a token
    query = [torch.randn((V, H, d), generator=g, device=DEV).bfloat16() for _ in range(2)]
    make = lambda: ([paged.PagedCache.new(60, page, d, fmt) for _ in range(2)],  # noqa: E731
                    layers.PagedState(ints([0] * B), ints(np.full((B, W), -1)), ints(range(60)), ints([60])))
    caches, state = make()
    plain, plain_state = make()

    def inputs(tokens, delta, k):
        t = torch.tensor(tokens, device=DEV)
        return layers.PagedInput(query[k][t], rows[k][t], ints(delta), cs)

    prompt = [50, 3, 70]
    tokens = r.integers(0, V, sum(prompt)).tolist()
    for c, s in ((caches, state), (plain, plain_state)):
        first = layers.paged_layer(c[0], s, inputs(tokens, prompt, 0), window, dv)
        layers.paged_layer_again(c[1], s, inputs(tokens, prompt, 1), first.plan, window, dv)
    last = r.integers(0, V, B).tolist()
    kept_all = 0
    for step in range(6):
        sizes = [int(r.integers(1, 12)) for _ in range(B)]
        sizes[0] = 12
        parent = [p for n in sizes for p in random_tree(r, n)]
        cu = np.cumsum([0] + sizes).tolist()
        tokens = r.integers(0, V, sum(sizes)).tolist()
        for b in range(B):
            tokens[cu[b]] = last[b]
        st = status()
        plan = layers.draft_plan(page, state, inputs(tokens, sizes, 0), ints(parent), 12, d_status=st)
        outs = [layers.draft_layer(caches[k], state, inputs(tokens, sizes, k), plan, window, dv, d_status=st) for k in range(2)]
        p = torch.softmax(torch.randn((sum(sizes), V), generator=g, device=DEV) * 2, 1)
        for b in range(B):                                                  # some drafts that stay
            for i in range(1, sizes[b]):
                if r.random() < 0.6:
                    p[cu[b] + parent[cu[b] + i], tokens[cu[b] + i]] += 1.0
        p /= p.sum(1, keepdim=True)
        v = draft.tree_verify(p, ints(tokens), ints(parent), plan.plan.cu, torch.rand(sum(sizes), generator=g, device=DEV),
                              torch.rand(B, generator=g, device=DEV), max_path=12, d_status=st)
        layers.draft_accept(caches, state, plan, v, d_status=st)
        assert int(st) == 0
        keep, path = v.keep.tolist(), v.path.tolist()
        kept_all += sum(keep) - B
        ways_ = [[cu[b] + i for i in path[b][:keep[b]]] for b in range(B)]
        # one after another
        for i in range(max(keep)):
            now = [w[i] for w in ways_ if i < len(w)]
            delta = [int(i < len(w)) for w in ways_]
            one = layers.paged_layer(plain[0], plain_state, inputs([tokens[t] for t in now], delta, 0), window, dv)
            two = layers.paged_layer_again(plain[1], plain_state, inputs([tokens[t] for t in now], delta, 1), one.plan, window, dv)
            for k, res in enumerate((one, two)):
                # both are within the bound of half a step each (weights and result rounded to bf16) of the same values
                got, want = outs[k].out[now].double(), res.out.double()
                assert float((got - want).abs().max()) <= 4 * 2.0 ** -8 * float(want.abs().max()) + 1e-6
                assert float((outs[k].lse[now] - res.lse).abs().max()) <= 1e-4
        last = v.token.tolist()
        assert state.lens.tolist() == plain_state.lens.tolist() and int(state.n_free) == int(plain_state.n_free)
        n = state.lens.tolist()
        for a, z in zip(caches, plain):
            for b in range(B):
                for x, y in zip(raw(a), raw(z)):
                    pa, pz = (s.block_table[b, :-(-n[b] // page)].cpu().numpy() for s in (state, plain_state))
                    assert np.array_equal(x[pa].reshape(-1, x.shape[2])[:n[b]], y[pz].reshape(-1, y.shape[2])[:n[b]])
    assert kept_all > 6


def test_answers_to_one_prompt():
    """A prompt forked three ways: each answer attends the prompt's rows and its own, as a request of its own would."""
    H, d, page, W, fmt = 16, 128, 16, 12, paged.MXFP4
    g, cs = torch.Generator(device=DEV).manual_seed(1), cos_sin(200, 32)
    x, q = torch.randn((90, d), generator=g, device=DEV).bfloat16(), torch.randn((90, H, d), generator=g, device=DEV).bfloat16()
    cache, alone = paged.PagedCache.new(40, page, d, fmt), paged.PagedCache.new(40, page, d, fmt)
    shared = layers.PagedState(ints([0] * 4), ints(np.full((4, W), -1)), ints(range(40)), ints([40]))
    own = layers.PagedState(ints([0] * 4), ints(np.full((4, W), -1)), ints(range(40)), ints([40]))
    shares = ints([0] * 40)
    layers.paged_layer(cache, shared, layers.PagedInput(q[:41], x[:41], ints([41, 0, 0, 0]), cs), d_v=d)
    layers.paged_layer(alone, own, layers.PagedInput(q[:41].repeat(4, 1, 1), x[:41].repeat(4, 1), ints([41] * 4), cs), d_v=d)
    st = status()
    args = (shared.lens, shared.block_table, shares, shared.free_pages, shared.n_free, page)
    f = draft.page_fork(ints([-1, 0, 0, 0]), *args, d_status=st)
    draft.page_copy([cache], f.src, f.dst, f.rows, d_status=st)
    assert int(shared.n_free) == 40 - 3 - 3 and int(own.n_free) == 40 - 12
    for step in range(9):
        at = slice(41 + 4 * step, 45 + 4 * step)
        a, z = (layers.paged_layer(c, s, layers.PagedInput(q[at], x[at], ints([1] * 4), cs), d_v=d, d_status=st) for c, s in ((cache, shared), (alone, own)))
        assert torch.equal(a.out, z.out) and torch.equal(a.lse, z.lse)
        if step == 4:
            draft.page_free(ints([1, 0, 1, 0]), *args, d_status=st)           # the prompt's own request ends before the others
            paged.page_plan(own.lens, ints([-46, 0, -46, 0]), own.block_table, own.free_pages, own.n_free, page, 0, in_place=True)
    assert int(st) == 0
    draft.page_free(ints([1] * 4), *args)
    assert sorted(shared.free_pages.tolist()) == list(range(40)) and int(shared.n_free) == 40
