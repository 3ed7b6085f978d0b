"""The paged-cache calls on the GPU against plain implementations in whole numbers and in 64 bits."""
import math

import numpy as np
import pytest
import torch

import oracle
from fp4_kv_cache_gb300 import csa2, layers, paged

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
I32 = torch.int32
FMTS = [paged.MXFP4, paged.NVFP4_E4M3_16, paged.MXFP8, paged.BF16]


def ints(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def status():
    return torch.zeros(1, dtype=I32, device=DEV)


# ------------------------------------------------------------------ bookkeeping
def plan_ref(lens, delta, table, free, n_free, page, n_rows):
    """The step request by request, with a list as the free stack."""
    B, W = table.shape
    table, stack, st = table.copy(), [int(v) for v in free[:max(n_free, 0)]], 0
    old = [max(int(v), 0) for v in lens]
    new = [min(max(o + int(d), 0), 2**31 - 1) for o, d in zip(old, delta)]
    had = [min(-(-o // page), W) for o in old]
    has = [min(-(-n // page), W) for n in new]
    for b in range(B):
        stack += [int(table[b, j]) for j in range(has[b], had[b])]
        if -(-new[b] // page) > W:
            st |= paged.DEV_TABLE_FULL
    for b in range(B):
        for j in range(had[b], has[b]):
            if not stack:
                st |= paged.DEV_NO_PAGES
            table[b, j] = stack.pop() if stack else -1
    cu = [0]
    rows = np.full((3, n_rows), -1, dtype=np.int64)
    for b in range(B):
        for i in range(max(new[b] - old[b], 0)):
            r, pos = cu[b] + i, old[b] + i
            if r >= n_rows:
                st |= paged.DEV_ROWS
                break
            j = pos // page
            slot = int(table[b, j]) * page + pos % page if j < W and table[b, j] >= 0 else -1
            rows[:, r] = slot, b, pos
        cu.append(cu[-1] + max(new[b] - old[b], 0))
    if len(stack) > len(free):
        st |= paged.DEV_TABLE_FULL
    left = min(len(stack), len(free))
    out_free = free.copy()
    out_free[:left] = stack[:left]
    return new, cu, rows, table, out_free, left, st


def plan_case(B, page, W, free_cap, max_len, max_new, drop, seed, shortage=0):
    r = np.random.default_rng(seed)
    lens = r.integers(0, max_len + 1, B)
    delta = np.where(r.random(B) < drop, -np.minimum(lens, r.choice([1, 3, 10**9], B)), r.integers(0, max_new + 1, B))
    held = np.minimum(-(-lens // page), W)
    need = int(held.sum())
    ids = r.permutation(need + free_cap).astype(np.int64)
    table = np.full((B, W), -7, dtype=np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(free_cap + need, -9, dtype=np.int64)
    n_free = max(free_cap - shortage, 0)
    free[:n_free] = ids[need:need + n_free]
    return lens, delta, table, free, n_free


@pytest.mark.parametrize("B,page,W,free_cap,max_len,max_new,drop,n_rows,shortage", [
    (1, 64, 4, 4, 100, 1, 0.0, 1, 0),
    (0, 64, 4, 4, 100, 1, 0.0, 5, 0),                 # no request: every row -1
    (7, 1, 40, 300, 30, 5, 0.3, 40, 0),               # a page a row
    (33, 16, 20, 700, 200, 70, 0.3, 1500, 0),
    (33, 16, 20, 40, 200, 70, 0.1, 2000, 20),         # the pages run out
    (9, 16, 5, 100, 80, 70, 0.2, 500, 0),             # tables too narrow
    (50, 32, 20, 600, 300, 100, 0.2, 700, 0),         # more rows than the slot map holds
    (600, 64, 40, 3000, 2000, 1, 0.0, 600, 0),
    (40, 64, 80, 3000, 3000, 2000, 0.4, 40001, 0),    # many rows: several CTAs
    (40, 64, 80, 200, 3000, 2000, 0.4, 40001, 100),   # ... and the pages run out
    (5003, 16, 12, 12000, 100, 20, 0.3, 60000, 0),
    (12, 16, 20, 200, 200, 0, 1.0, 16, 0),            # everything is given back
])
def test_page_plan(B, page, W, free_cap, max_len, max_new, drop, n_rows, shortage):
    lens, delta, table, free, n_free = plan_case(B, page, W, free_cap, max_len, max_new, drop, B + n_rows, shortage)
    ref = plan_ref(lens, delta, table, free, n_free, page, n_rows)
    st = status()
    t_table, t_free, t_lens, t_n = ints(table.reshape(B, W)), ints(free), ints(lens), ints([n_free])
    p = paged.page_plan(t_lens, ints(delta), t_table, t_free, t_n, page, n_rows, d_status=st)
    assert p.lens.tolist() == ref[0] and p.cu.tolist() == ref[1]
    for got, want in zip((p.slot, p.row_req, p.row_pos), ref[2]):
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(t_table.cpu().numpy(), ref[3])
    left = ref[5]
    assert int(p.n_free) == left and np.array_equal(t_free.cpu().numpy()[:left], ref[4][:left])
    assert np.array_equal(t_free.cpu().numpy()[max(left, n_free):], free[max(left, n_free):])
    assert int(st) == ref[6]
    assert t_lens.tolist() == list(lens) and int(t_n) == n_free


def test_page_plan_negative_and_huge_lengths():
    st = status()
    table, free = ints([[3, 4], [5, 6], [7, 8]]), ints([9, 10, 11])
    p = paged.page_plan(ints([-5, 20, 2**31 - 1]), ints([4, -100, 100]), table, free, ints([3]), 16, 8, d_status=st)
    assert p.lens.tolist() == [4, 0, 2**31 - 1]
    assert p.slot.tolist()[:4] == [6 * 16 + i for i in range(4)]           # the last page given back is on top
    assert p.cu.tolist() == [0, 4, 4, 4] and p.slot.tolist()[4:] == [-1] * 4
    # four pages are free then, and the list holds three
    assert int(p.n_free) == 3 and free.tolist() == [9, 10, 11]
    assert int(st) == paged.DEV_TABLE_FULL


def test_page_plan_replayed_in_place():
    # a captured step: lengths, count, table and free list carry over, delta changes
    B, page, W = 5, 4, 16
    lens, table, free, n_free = ints([0] * B), ints(np.full((B, W), -1)), ints(range(80)), ints([80])
    delta = ints([1] * B)
    buf = torch.empty(64, dtype=I32, device=DEV)
    plan = paged.PagePlan(lens, buf[:B + 1], buf[8:18], buf[20:30], buf[32:42], n_free)
    rl, rt, rf, rn = np.zeros(B, int), table.cpu().numpy().astype(np.int64), free.cpu().numpy().astype(np.int64), 80
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        delta.zero_()
        paged.page_plan(lens, delta, table, free, n_free, page, 10, plan=plan)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paged.page_plan(lens, delta, table, free, n_free, page, 10, plan=plan)
    for d in ([1, 1, 1, 1, 1], [2, 0, 3, 1, 4], [-2, 5, -1, 0, 3], [1, -4, 2, 2, -100], [9, 0, 0, 0, 1]):
        delta.copy_(ints(d))
        g.replay()
        new, cu, rows, rt, rf, rn, _ = plan_ref(rl, d, rt, rf, rn, page, 10)
        rl = np.array(new)
        assert lens.tolist() == new and plan.cu.tolist() == cu and int(n_free) == rn
        assert plan.slot.tolist() == rows[0].tolist() and np.array_equal(table.cpu().numpy(), rt)
        assert free.tolist()[:rn] == rf[:rn].tolist()


# ------------------------------------------------------------------ rotation
def cos_sin(n_pos, rope):
    f = 10000.0 ** (-np.arange(0, rope, 2) / rope)
    a = np.arange(n_pos)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(DEV)


def turned32(x, pos, cs, sections):
    """x float32 [..., d] turned with one rounding per product and sum; pos [axes, rows]."""
    y, half = x.clone(), cs.shape[1] // 2
    i = 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            p = pos[axis].long()
            ok = (p >= 0) & (p < cs.shape[0])
            p = p.clamp(0, cs.shape[0] - 1)
            c, s = torch.where(ok, cs[p, i], 1.0), torch.where(ok, cs[p, half + i], 0.0)
            c, s = (t.view((-1,) + (1,) * (x.dim() - 2)) for t in (c, s))
            k = x.shape[-1] - 2 * half + 2 * i
            a, b = x[..., k], x[..., k + 1]
            y[..., k], y[..., k + 1] = a * c - b * s, a * s + b * c
            i += 1
    return y


@pytest.mark.parametrize("rows,heads,d,rope,sections", [
    (1, 1, 8, 2, [1]), (3, 5, 64, 64, [32]), (17, 64, 576, 64, [32]), (200, 16, 128, 32, [4, 6, 6]), (33, 8, 576, 64, [0, 20, 12]),
    (5, 3, 72, 36, [9, 9]), (7, 2, 576, 0, None), (2100, 2, 40, 6, [1, 1, 1])])
@pytest.mark.parametrize("how", ["new", "place", "strided"])
def test_rope(rows, heads, d, rope, sections, how):
    g = torch.Generator(device=DEV).manual_seed(rows * d)
    wide = torch.randn((rows, heads + 1, d + 8), generator=g, device=DEV).bfloat16()
    x = wide[:, 1:, 8:] if how == "strided" else wide[:, 1:, 8:].contiguous()
    keep = x.clone()
    axes = len(sections) if sections else 1
    pos = torch.randint(0, 4000, (axes, rows), generator=g, device=DEV, dtype=I32)
    cs = cos_sin(4000, rope) if rope else None
    want = turned32(x.float(), pos, cs, sections).bfloat16() if rope else x.clone()
    st = status()
    args = (pos if axes > 1 else pos[0], cs, sections) if rope else (None, None, None)
    out = paged.rope_axes(x, *args, out=x if how != "new" else None, d_status=st)
    assert torch.equal(out, want) and int(st) == 0
    if how == "new":
        assert torch.equal(x, keep)
    if how == "strided":
        assert out.data_ptr() == x.data_ptr()


def test_rope_bad_positions():
    x, cs = torch.randn((4, 3, 64), device=DEV).bfloat16(), cos_sin(100, 32)
    for last, want in ((99, 0), (100, csa2.DEV_BAD_INDEX)):               # below 0: nothing to turn
        pos, st = ints([[0, -1, 99, 3], [5, 2, last, -2**31]]), status()
        out = paged.rope_axes(x, pos, cs, [10, 6], d_status=st)
        assert torch.equal(out, turned32(x.float(), pos, cs, [10, 6]).bfloat16())
        assert int(st) == want


# ------------------------------------------------------------------ write and read
def quantised(y, fmt):
    """Oracle codes and scales of float32 rows."""
    f = {paged.MXFP4: oracle.quant_mxfp4, paged.NVFP4_E4M3_16: oracle.quant_nvfp4, paged.MXFP8: oracle.quant_mxfp8}[fmt]
    return f(y.cpu().numpy())


def values64(codes, scales, fmt):
    """Values of rows of codes in 64 bits."""
    if fmt == paged.BF16:
        return codes.double()
    c = codes.long()
    if fmt == paged.MXFP8:
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m / 512)
        v = torch.where((c & 127) == 127, math.nan, v) * (1.0 - 2.0 * (c >> 7))
    else:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e > 0, (2 + m) * torch.exp2((e - 2).double()), m / 2) * (1.0 - 2.0 * (c >> 3))
    s = scales.long()
    if fmt == paged.NVFP4_E4M3_16:
        e, m = (s >> 3) & 15, (s & 7).double()
        sc = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m / 512)
        sc = torch.where((s & 127) == 127, math.nan, sc) * (1.0 - 2.0 * (s >> 7))
    else:
        sc = torch.where(s == 255, math.nan, torch.exp2((s - 127).double()))
    return v * sc.repeat_interleave(16 if fmt == paged.NVFP4_E4M3_16 else 32, -1)


def strided_cache(n_pages, page, d, fmt, layers_=3):
    """A cache whose pages lie between other layers' pages, all bytes random."""
    g = torch.Generator(device=DEV).manual_seed(n_pages)
    shape = paged.PagedCache.new(1, 1, d, fmt, device="cpu")
    codes = torch.randint(0, 255, (n_pages, layers_, page, shape.codes.shape[2]), generator=g, device=DEV, dtype=torch.uint8)
    if fmt == paged.BF16:
        codes = codes.to(torch.bfloat16)
        return codes, None, paged.PagedCache(codes[:, 1])
    scales = torch.randint(100, 140, (n_pages, layers_, page, shape.scales.shape[2]), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales, paged.PagedCache(codes[:, 1], scales[:, 1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,d,page,rope,sections", [
    (1, 32, 1, 0, None), (37, 576, 16, 64, [32]), (300, 128, 64, 32, [4, 6, 6]), (65, 512, 128, 512, [100, 156]), (9, 1024, 2, 6, [3])])
def test_write_and_read(fmt, rows, d, page, rope, sections):
    g = torch.Generator(device=DEV).manual_seed(rows + d + fmt)
    x = (torch.randn((rows, d + 8), generator=g, device=DEV)
         * torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g, device=DEV).float())).bfloat16()[:, 8:]
    x[0, ::3] = 0.0
    x[rows // 2, :32] = -0.0
    n_pages = -(-rows // page) + 2
    codes, scales, cache = strided_cache(n_pages, page, d, fmt)
    before = codes.clone(), scales.clone() if scales is not None else None
    slot = torch.randperm(n_pages * page, generator=g, device=DEV)[:rows].to(I32)
    if rows > 4:
        slot[3] = -1                                                        # not written
    axes = len(sections) if sections else 1
    pos = torch.randint(0, 900, (axes, rows), generator=g, device=DEV, dtype=I32)
    cs = cos_sin(900, rope) if rope else None
    st = status()
    paged.paged_write(cache, x, slot, *((pos if axes > 1 else pos[0], cs, sections) if rope else ()), d_status=st)
    y = turned32(x.float(), pos, cs, sections) if rope else x.float()
    at = slot.long()
    ok = at >= 0
    pg, off = at[ok] // page, at[ok] % page
    want = before
    if fmt == paged.BF16:
        want[0][pg, 1, off] = y[ok].bfloat16()
    else:
        c, s = quantised(y[ok], fmt)
        want[0][pg, 1, off] = torch.from_numpy(c).to(DEV)
        want[1][pg, 1, off] = torch.from_numpy(s).to(DEV)
        assert torch.equal(scales, want[1])
    assert torch.equal(codes, want[0])                                      # nothing else was touched
    assert int(st) == 0
    out = torch.full((rows, d + 16), 7.0, dtype=torch.bfloat16, device=DEV)[:, 8:d + 8]
    paged.paged_read(cache, slot, out=out, d_status=st)
    v = values64(cache.codes[pg, off], cache.scales[pg, off] if scales is not None else None, fmt).bfloat16()
    assert torch.equal(out[ok], v) and bool((out[~ok] == 7.0).all()) and int(st) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_write_and_read_bad_slots_and_values(fmt):
    cache = paged.PagedCache.new(4, 16, 64, fmt)
    x, st = torch.full((5, 64), 6.0, dtype=torch.bfloat16, device=DEV), status()
    slot = ints([0, 64, -1, 63, 2**31 - 1])
    paged.paged_write(cache, x, slot, d_status=st)
    assert int(st) == csa2.DEV_BAD_INDEX
    assert int((paged.paged_read(cache, ints(range(64))).sum(1) > 0).sum()) == 2
    st = status()
    out = torch.zeros((5, 64), dtype=torch.bfloat16, device=DEV)
    paged.paged_read(cache, slot, out=out, d_status=st)
    assert out.float().sum(1).tolist() == [384.0, 0.0, 0.0, 384.0, 0.0] and int(st) == csa2.DEV_BAD_INDEX
    x[1, 40], st = math.inf, status()
    paged.paged_write(cache, x, ints([5, 6, 7, 8, 9]), d_status=st)
    assert int(st) == (0 if fmt == paged.BF16 else csa2.DEV_NONFINITE)
    assert bool((paged.paged_read(cache, ints([5, 7, 5])) == 6.0).all())     # the rows beside it, one of them twice


# ------------------------------------------------------------------ attention
def random_cache(n_pages, page, d, fmt, seed, scale=1.0):
    """Rows of normal values, written through the library's contiguous codecs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = paged.PagedCache.new(n_pages, page, d, fmt)
    step = max(1, (1 << 25) // (page * d))
    for at in range(0, n_pages, step):
        n = min(step, n_pages - at)
        x = torch.randn((n, page, d), generator=g, device=DEV) * scale
        if fmt == paged.BF16:
            c.codes[at:at + n] = x.bfloat16()
        else:
            cc, ss = csa2.quant_fp8(x) if fmt == paged.MXFP8 else csa2.quant_fp4(x, fmt=fmt)
            c.codes[at:at + n], c.scales[at:at + n] = cc, ss
    return c


class AttnCase:
    def __init__(self, lens, new, H, d, dv, fmt, page, window=0, ratio=1, pos0=None, start=None, seed=0, q_scale=1.0, pad=0, kv_scale=1.0):
        self.g = torch.Generator(device=DEV).manual_seed(seed + 100)
        self.lens, self.new, self.H, self.d, self.dv, self.window, self.ratio = lens, new, H, d, dv, window, ratio
        need = [-(-n // page) for n in lens]
        self.cache = random_cache(sum(need) + 3, page, d, fmt, seed, kv_scale)
        order = torch.randperm(sum(need) + 3, generator=self.g, device=DEV).tolist()
        self.table = np.full((len(lens), max(need + [0]) + 2), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        T = sum(new) + pad
        self.q = (torch.randn((T, H, d), generator=self.g, device=DEV) * q_scale).bfloat16()
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.pos0 = pos0
        self.start = start
        self.sm = 1.0 / math.sqrt(d)

    def run(self, st=None, stream=None, **k):
        opt = dict(pos0=ints(self.pos0) if self.pos0 is not None else None, kv_start=ints(self.start) if self.start is not None else None)
        opt.update(k)
        table = torch.from_numpy(self.table).to(DEV).to(I32)
        return paged.paged_attn(self.q, self.cache, table, ints(self.lens), ints(self.cu), d_v=self.dv, window=self.window,
                                ratio_m=self.ratio, sm_scale=self.sm, d_status=st, stream=stream, **opt)

    def ref(self):
        """(out, lse, bound of out, bound of lse) in 64 bits, tokens outside every request left zero."""
        page, T = self.cache.page, self.q.shape[0]
        out = torch.zeros((T, self.H, self.dv), dtype=torch.float64, device=DEV)
        lse = torch.full((T, self.H), -math.inf, dtype=torch.float64, device=DEV)
        ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
        for b, n in enumerate(self.lens):
            t0, t1 = int(self.cu[b]), int(self.cu[b + 1])
            if t1 <= t0:
                continue
            pages = torch.from_numpy(self.table[b, :-(-n // page)]).to(DEV)
            good = ((pages >= 0) & (pages < self.cache.n_pages)).repeat_interleave(page)[:n]
            pages = pages.clamp(0, self.cache.n_pages - 1)
            k = values64(self.cache.codes[pages].flatten(0, 1)[:n],
                         self.cache.scales[pages].flatten(0, 1)[:n] if self.cache.scales is not None else None, self.cache.fmt)
            p = (self.pos0[b] if self.pos0 is not None else n - (t1 - t0)) + torch.arange(t1 - t0, device=DEV)
            e = torch.div((p + 1).clamp(min=0), self.ratio, rounding_mode="floor")
            lo = torch.zeros_like(e) if self.start is None else torch.full_like(e, self.start[b])
            if self.window:
                lo = torch.maximum(lo, e - self.window)
            j = torch.arange(n, device=DEV)
            see = (j < e[:, None]) & (j >= lo[:, None]) & good
            q = self.q[t0:t1].double()
            bad = ~torch.isfinite(k).all(1)                                # rows that poison who sees them
            kz = torch.where(bad[:, None], 0.0, k)
            z = torch.einsum("thd,jd->thj", q, kz) * self.sm
            z = z.masked_fill(~see[:, None], -math.inf)
            top = z.amax(-1) if n else torch.full((t1 - t0, self.H), -math.inf, dtype=torch.float64, device=DEV)
            some = top > -math.inf
            w = torch.exp(z - torch.where(some, top, 0.0)[..., None])
            tot = w.sum(-1)
            w = w / torch.where(some, tot, 1.0)[..., None]
            nan = (see & bad).any(1)
            o = w @ kz[:, :self.dv]
            o[nan] = math.nan
            out[t0:t1] = o
            lse[t0:t1] = torch.where(some, top + torch.log(torch.where(some, tot, 1.0)), -math.inf)
            lse[t0:t1][nan] = math.nan
            # logits: d products of bf16 values summed in float32 (any order), each sum off by at most
            # 2^-23 of the sum of magnitudes, then scaled, subtracted and raised with 2^-22 each; a
            # weight is then rounded to bf16 (2^-8 of it at most) and so is the result
            mag = torch.einsum("thd,jd->thj", q.abs(), kz.abs()).masked_fill(~see[:, None], 0.0).amax(-1) * self.sm if n else torch.zeros_like(tot)
            dl = mag * self.d * 2.0 ** -23 + 2.0 ** -20 + torch.where(some, top.abs(), 0.0) * 2.0 ** -21
            a = w @ kz[:, :self.dv].abs()
            ob[t0:t1] = o.abs() * 2.0 ** -8 + a * (2.0 ** -8 + 2 * dl[..., None] + n * 2.0 ** -23) * 1.01 + 1e-30
            lb[t0:t1] = dl * 1.01 + n * 2.0 ** -23 + 2.0 ** -20
        return out, lse, ob, lb


def close(got, want, bound):
    got = got.double()
    same = torch.isnan(got) == torch.isnan(want)
    inf = torch.isinf(want)
    same &= torch.where(inf, got == want, True)
    fine = torch.isfinite(want)
    diff = torch.where(fine, (got - want).abs(), 0.0)
    worst = float((diff / bound.clamp(min=1e-300))[fine].max()) if bool(fine.any()) else 0.0
    assert bool(same.all()), f"{int((~same).sum())} values not finite where they should be, or the other way"
    assert worst <= 1.0, f"off by {worst:.3f} of the bound"


def check(case, st_want=0, **k):
    st = status()
    out, lse = case.run(st, **k)
    o, l, ob, lb = case.ref()
    n = int(case.cu[-1])
    close(out[:n], o[:n], ob[:n])
    close(lse[:n], l[:n], lb[:n])
    assert int(st) == st_want
    return out, lse


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,d,dv", [(64, 576, 512), (16, 128, 128), (1, 32, 8), (128, 512, 512), (5, 96, 40), (33, 288, 264),
                                    (48, 576, 520 - 8)])
def test_attn_formats_and_heads(fmt, H, d, dv):
    check(AttnCase([300, 1, 77], [3, 1, 5], H, d, dv, fmt, 16, seed=H + fmt))


@pytest.mark.parametrize("lens,new,page", [
    ([1], [1], 64), ([63], [1], 64), ([64], [1], 64), ([65], [1], 64), ([127], [2], 128), ([128], [2], 128), ([129], [3], 128),
    ([255, 256, 257], [1, 1, 1], 32), ([1000], [1], 1), ([513], [513], 16), ([5000, 3, 700], [1, 3, 40], 64),
    ([20000], [1], 64), ([20000, 19999], [2, 5], 256), ([130] * 40, [1] * 40, 64), ([7, 0, 9], [1, 0, 2], 8),
    ([4096], [200], 4096)])
def test_attn_lengths(lens, new, page):
    check(AttnCase(lens, new, 64, 576, 512, paged.MXFP4, page, seed=lens[0]))


@pytest.mark.parametrize("window,ratio,pos0,start", [
    (1, 1, None, None), (128, 1, None, None), (100, 1, None, [0, 290, 3]), (0, 2, [500, 0, 30], None), (60, 2, [598, 1, 99], [3, 0, 0]),
    (0, 1, [-3, -1, 200], None),              # queries before the first row, and past the last
    (0, 1, None, [300, 1000, 0]),             # rows that leave a token nothing
    (5, 1, [1000, 2**30, 2**31 - 8], None),   # windows past the cache
    (0, 4, [2**31 - 40, 3, 7], [-5, -1, 0])])
def test_attn_masks(window, ratio, pos0, start):
    check(AttnCase([300, 310, 200], [40, 3, 30], 16, 128, 128, paged.NVFP4_E4M3_16, 16, window, ratio, pos0, start, seed=window + ratio))


def test_attn_large_logits():
    # one weight holds almost everything; sums of large and small logits
    check(AttnCase([700, 300], [3, 20], 64, 576, 512, paged.MXFP4, 32, q_scale=30.0, seed=4))


def test_attn_small_logits():
    check(AttnCase([2000], [2], 64, 576, 512, paged.MXFP8, 32, q_scale=1e-3, seed=5))


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.MXFP8, paged.BF16])
@pytest.mark.parametrize("scale", [2.0 ** 30, 2.0 ** -40])
def test_attn_scales_of_rows(fmt, scale):
    # block scales far from one, where a short product range would overflow or vanish
    check(AttnCase([200], [4], 16, 128, 128, fmt, 32, q_scale=1.0 / scale, kv_scale=scale, seed=6))


@pytest.mark.parametrize("fmt,scale", [(paged.MXFP4, 4.0), (paged.MXFP8, 2.0 ** 14)])
def test_attn_scales_around_one_factor(fmt, scale):
    # block scales on both sides of the largest that one bf16 factor holds
    case = AttnCase([400], [4], 16, 576, 512, fmt, 32, q_scale=1.0 / scale, kv_scale=scale, seed=16)
    held = 128 if fmt == paged.MXFP4 else 134
    assert bool((case.cache.scales <= held).any()) and bool((case.cache.scales > held).any())
    check(case)


@pytest.mark.parametrize("window", [127, 128, 129, 255, 256, 257])
def test_attn_windows_around_tiles(window):
    check(AttnCase([1000, 130, 257], [5, 130, 1], 64, 576, 512, paged.MXFP8, 128, window=window, seed=window))


def test_attn_bad_pages():
    c = AttnCase([300, 400, 200], [4, 2, 3], 64, 576, 512, paged.MXFP4, 16, seed=7)
    c.table[0, 3], c.table[0, 18], c.table[1, 0], c.table[2, 1:] = -1, 2**31 - 1, c.cache.n_pages, -2**31
    check(c, csa2.DEV_BAD_INDEX)
    c = AttnCase([300], [4], 16, 128, 128, paged.MXFP4, 16, seed=8)
    c.table[:] = -1                                        # no row left at all
    out, lse = check(c, csa2.DEV_BAD_INDEX)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attn_length_past_the_table():
    c = AttnCase([300], [4], 16, 128, 128, paged.MXFP4, 16, pos0=[296], seed=9)
    want = c.run()[0]
    c.table = c.table[:, :19]
    c.lens = [10**6]                                       # rows 300.. are not in the table; none is visible
    st = status()
    assert torch.equal(c.run(st)[0], want) and int(st) == 0
    c.pos0 = [400]                                         # now some would be
    c.run(st)
    assert int(st) == csa2.DEV_BAD_INDEX


@pytest.mark.parametrize("fmt", FMTS)
def test_attn_not_finite_rows(fmt):
    # rows that are not finite: unseen ones (masked, past the length, in unused pages) change nothing,
    # a seen one makes its queries NaN and no others
    c = AttnCase([200, 150], [60, 60], 16, 128, 128, fmt, 16, seed=10)
    bad = [(0, 170), (1, 149)]
    dirty = [(0, 200), (0, 207), (1, 150), (1, 159)]
    for b, j in bad + dirty:
        pg, off = int(c.table[b, j // 16]), j % 16
        if fmt == paged.BF16:
            c.cache.codes[pg, off, 5] = math.inf if j % 2 else math.nan
        elif fmt == paged.MXFP8 and j % 2:
            c.cache.codes[pg, off, 100] = 0xFF
        else:
            c.cache.scales[pg, off, 1] = 0x7F if fmt == paged.NVFP4_E4M3_16 else 255
    out, _ = check(c)
    assert int(torch.isnan(out).any(-1).any(-1).sum()) == 30 + 1


def test_attn_queries_not_finite():
    c = AttnCase([200], [60], 16, 128, 128, paged.MXFP4, 16, seed=11)
    want, _ = c.run()
    c.q[7, 3, 100] = math.nan
    got, _ = c.run()
    same = torch.ones((60, 16), dtype=torch.bool, device=DEV)
    same[7, 3] = False
    assert torch.equal(got[same], want[same]) and bool(torch.isnan(got[7, 3]).all())


def test_attn_rows_outside_stay():
    c = AttnCase([100, 60], [3, 5], 16, 128, 128, paged.MXFP4, 16, seed=12, pad=9)
    out = torch.full((17, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((17, 16), 4.0, device=DEV)
    check(c, out=out, lse=lse)
    assert bool((out[8:] == 3.0).all()) and bool((lse[8:] == 4.0).all())
    c.cu = c.cu + 2                                        # and before the first request
    out.fill_(3.0), lse.fill_(4.0)
    c.run(out=out, lse=lse)
    assert bool((out[:2] == 3.0).all()) and bool((lse[:2] == 4.0).all()) and bool((out[10:] == 3.0).all())
    assert not bool((out[2:10] == 3.0).all(-1).any())


def test_attn_cu_past_the_queries():
    # offsets past n_tokens are left out, never read or written
    c = AttnCase([100, 60], [3, 5], 16, 128, 128, paged.MXFP4, 16, pos0=[97, 55], seed=13)
    want = c.run()[0]
    c.cu = np.array([0, 3, 500])
    assert torch.equal(c.run()[0][:3], want[:3])


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.NVFP4_E4M3_16])
def test_attn_strided_pages(fmt):
    c = AttnCase([300, 100], [5, 1], 64, 576, 512, fmt, 16, seed=14)
    want = c.run()
    n = c.cache.n_pages
    codes = torch.randint(0, 255, (n, 3, 16, 288), device=DEV, dtype=torch.uint8)
    scales = torch.full((n, 2, 16, c.cache.scales.shape[2]), 255, device=DEV, dtype=torch.uint8)
    codes[:, 2], scales[:, 1] = c.cache.codes, c.cache.scales
    c.cache = paged.PagedCache(codes[:, 2], scales[:, 1])
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_far_pages():
    # pages whose byte offsets pass 32 bits
    n, page, d = 2_100_000, 2, 576
    codes = torch.empty((n, page, d), dtype=torch.bfloat16, device=DEV)
    c = AttnCase([50], [3], 16, d, 512, paged.BF16, page, seed=15)
    want = c.run()
    far = torch.arange(n - c.cache.n_pages, n, device=DEV)
    codes[far] = c.cache.codes
    c.table = np.where(c.table >= 0, c.table + n - c.cache.n_pages, -1)
    c.cache = paged.PagedCache(codes)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_same_twice_and_workspace():
    # no atomics decide anything: the same inputs give the same bits, in a dirty workspace too
    c = AttnCase([9000, 40, 3000], [2, 30, 1], 64, 576, 512, paged.MXFP4, 64, seed=16)
    a = c.run()
    ws = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        b = c.run(workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attn_streams_and_graphs():
    # two calls at once on two streams, then both captured and replayed with new lengths
    cs = [AttnCase([6000, 500], [2, 30], 64, 576, 512, paged.MXFP4, 64, seed=s) for s in (17, 18)]
    want = [c.run() for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(c.run())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = cs[0]
    table, lens, cu = torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu)
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paged.paged_attn(c.q, c.cache, table, lens, cu, d_v=512, sm_scale=c.sm, out=out, lse=lse, workspace=ws)
    for new_lens in ([6000, 500], [40, 480], [5990, 31]):
        lens.copy_(ints(new_lens))
        c.lens = new_lens
        g.replay()
        o, l, ob, lb = c.ref()
        close(out, o, ob)
        close(lse, l, lb)


def test_attn_given_stream():
    c = AttnCase([3000], [5], 64, 576, 512, paged.MXFP4, 64, seed=19)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_given_stream_owns_what_a_call_allocates():
    # a block that the current stream still writes is not handed to the other stream's call
    x = torch.randn((512, 8, 128), device=DEV).bfloat16()
    cs, pos = cos_sin(600, 32), ints(range(512))
    want = paged.rope_axes(x, pos, cs)
    s, big = torch.cuda.Stream(), torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        busy = torch.empty_like(want)
        for _ in range(20):
            big = torch.tanh(big @ big)
        busy.fill_(7.0)
        del busy
        got = paged.rope_axes(x, pos, cs, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_attn_refuses_workspace():
    c = AttnCase([300], [2], 16, 128, 128, paged.MXFP4, 32, seed=20)
    with pytest.raises(ValueError):
        c.run(workspace=torch.empty(1 << 26, dtype=torch.uint8))
    with pytest.raises(ValueError):
        c.run(workspace=torch.empty((2, 1 << 26), dtype=torch.uint8, device=DEV)[:, ::2])
    with pytest.raises(paged.Csa2Error):
        c.run(workspace=torch.empty(1024, dtype=torch.uint8, device=DEV))


def test_attn_overlapping_requests():
    # bounds that give the same rows to two requests: flagged, nothing written
    c = AttnCase([40, 7, 33], [5, 0, 0], 64, 128, 128, paged.MXFP4, 32, seed=21)
    c.cu = np.array([0, 5, 0, 5])
    out = torch.full((5, 64, 128), 3.0, device=DEV).bfloat16()
    lse = torch.full((5, 64), 3.0, device=DEV)
    st = status()
    c.run(st, out=out, lse=lse)
    assert int(st) == csa2.DEV_BAD_INDEX
    assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt", [paged.NVFP4_E4M3_16, paged.MXFP8])
def test_steps_of_a_server(fmt):
    """Prompts, chunks, decode steps, drafts taken back and an ended request through layers.paged_layer."""
    H, d, dv, rope, page, W, B = 16, 128, 128, 32, 16, 20, 4
    g = torch.Generator(device=DEV).manual_seed(fmt)
    cache = paged.PagedCache.new(60, page, d, fmt)
    state = layers.PagedState(ints([0] * B), ints(np.full((B, W), -1)), ints(range(60)), ints([60]))
    cs, kept = cos_sin(400, rope), [torch.zeros((0, d), device=DEV) for _ in range(B)]
    for step, delta in enumerate(([100, 3, 0, 61], [1, 1, 40, 1], [1, -2, 1, 1], [30, 1, 1, -10**6], [5, 5, 5, 5])):
        n = sum(max(v, 0) for v in delta)
        pad = 3
        x = torch.randn((n + pad, d), generator=g, device=DEV).bfloat16()
        q = torch.randn((n + pad, H, d), generator=g, device=DEV).bfloat16()
        st = status()
        out = layers.paged_layer(cache, state, layers.PagedInput(q, x, ints(delta), cs), d_v=dv, window=70 if step == 3 else 0, d_status=st)
        assert int(st) == 0
        first, lens = 0, []
        for b, v in enumerate(delta):
            if v < 0:
                kept[b] = kept[b][:max(0, kept[b].shape[0] + v)]
            old = kept[b].shape[0]
            pos = torch.arange(old, old + max(v, 0), device=DEV)[None].to(I32)
            y = turned32(x[first:first + max(v, 0)].float(), pos, cs, [rope // 2])
            if v > 0:
                codes, scales = (torch.from_numpy(t).to(DEV) for t in quantised(y, fmt))
                kept[b] = torch.cat([kept[b], values64(codes, scales, fmt).float()])
            lens.append(kept[b].shape[0])
            qr = turned32(q[first:first + max(v, 0)].float(), pos, cs, [rope // 2]).bfloat16().double()
            for t in range(max(v, 0)):
                k = kept[b][max(0, old + t + 1 - 70) if step == 3 else 0:old + t + 1].double()
                z = qr[t] @ k.T / math.sqrt(d)
                ref = torch.softmax(z, -1) @ k[:, :dv]
                # rounding of weights and result, 2^-8 each, and slack for the float32 sums
                bound = ref.abs() * 2.0 ** -8 + (torch.softmax(z, -1) @ k[:, :dv].abs()) * (2.0 ** -8 + 2.0 ** -12)
                close(out.out[first + t], ref, bound)
            first += max(v, 0)
        assert state.lens.tolist() == lens and int(state.n_free) == 60 - sum(-(-v // page) for v in lens)


def test_paged_is_sparse_attention_of_everything():
    # a selection of every row, and no window, is the same attention
    c = AttnCase([400], [1], 64, 576, 512, paged.MXFP4, 16, seed=20)
    out, lse = c.run()
    pages = torch.from_numpy(c.table[0, :25]).to(DEV)
    idx = torch.arange(400, device=DEV, dtype=I32)[None, None]
    o2, l2 = csa2.sparse_attn(c.q[None], c.cache.codes[pages].flatten(0, 1)[None].contiguous(),
                              c.cache.scales[pages].flatten(0, 1)[None].contiguous(), idx, d_v=512, sm_scale=c.sm)
    _, _, ob, lb = c.ref()
    close(o2[0], out.double(), 2 * ob)
    close(l2[0], lse.double(), 2 * lb)
