"""Paged-cache calls at their edges: steps after a shortage of pages, offsets that step down or leave
the queries, masks that leave leading pages unread, rows that are not finite, calls at once."""
import math
import threading

import numpy as np
import pytest
import torch

from fp4_kv_cache_gb300 import csa2, layers, paged
from test_gpu_paged import AttnCase, DEV, FMTS, I32, check, close, cos_sin, ints, status, turned32, values64
from test_paged_refusals import strides

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ bookkeeping
def plan_step(lens, delta, table, stack, page):
    """One step on lists: lens and table are updated, the stack of free pages is popped and pushed."""
    new = [max(n + d, 0) for n, d in zip(lens, delta)]
    had, has = ([-(-n // page) for n in v] for v in (lens, new))
    for row, a, z in zip(table, has, had):
        stack += [p for p in row[a:max(a, z)] if p >= 0]
    short = False
    for row, a, z in zip(table, had, has):
        for j in range(a, z):
            short |= not stack
            row[j] = stack.pop() if stack else -1
    slots = [row[p // page] * page + p % page if row[p // page] >= 0 else -1
             for row, n, m in zip(table, lens, new) for p in range(n, m)]
    lens[:] = new
    return slots, paged.DEV_NO_PAGES if short else 0


def run_plan(steps, lens, table, free, n_pages, page, n_rows, in_place):
    """The steps on the GPU beside plan_step; every page stays either free or in one table."""
    width = len(table[0])
    t_lens, t_table, t_n = ints(lens), ints(table), ints([len(free)])
    t_free = ints(free + [-9] * (n_pages - len(free)))
    for delta in steps:
        before, st = list(lens), status()
        slots, want = plan_step(lens, delta, table, free, page)
        p = paged.page_plan(t_lens, ints(delta), t_table, t_free, t_n, page, n_rows, in_place=in_place, d_status=st)
        assert int(st) == want and p.lens.tolist() == lens
        assert t_table.tolist() == table and int(p.n_free) == len(free) and t_free.tolist()[:len(free)] == free
        assert p.slot.tolist() == slots + [-1] * (n_rows - len(slots))
        held = [v for row, n in zip(table, lens) for v in row[:-(-n // page)] if v >= 0]
        assert sorted(held + free) == list(range(n_pages))
        if in_place:
            assert t_lens.tolist() == lens and int(t_n) == len(free)
        else:
            assert t_lens.tolist() == before
            t_lens, t_n = p.lens.clone(), p.n_free.clone()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_rows", [8, 5000])                             # one CTA, and several
def test_plan_after_a_shortage(n_rows, in_place):
    # a request starves, is taken back, and another asks: it gets the page that is free
    run_plan([[0, 8], [0, -8], [0, 4], [-4, 0], [8, 0]], [4, 0], [[0, -1, -1], [-1, -1, -1]], [1], 2, 4, n_rows, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,n_pages,most,n_rows,seed", [
    (3, 4, 6, 12, 64, 0), (9, 1, 60, 40, 400, 1), (9, 4, 90, 300, 3000, 2), (70, 16, 200, 400, 30000, 3), (700, 2, 900, 9, 7000, 4),
    (40, 1, 900, 200, 8000, 5)])
def test_plan_steps_with_shortages(B, page, n_pages, most, n_rows, seed, in_place):
    # too few pages all the time: requests grow past the free list, shrink across its holes and end
    r = np.random.default_rng(seed)
    lens, steps = [0] * B, []
    for _ in range(12):
        grow = r.integers(0, most + 1, B)
        back = -np.minimum(lens, r.choice([1, page + 1, most // 2 + 1, 10**6], B))
        d = np.where(r.random(B) < 0.4, back, np.where(np.array(lens) > 3 * most, 0, grow))
        steps.append([int(v) for v in d])
        lens = [n + int(v) for n, v in zip(lens, d)]
    width = 4 * most // page + 2
    run_plan(steps, [0] * B, [[-1] * width for _ in range(B)], list(range(n_pages)), n_pages, page, n_rows, in_place)


@pytest.mark.parametrize("own_lens", [False, True])
def test_plan_of_several_ctas_captured(own_lens):
    # replayed with new deltas, pages running out on the way: lengths (or not) and count overwrite the old ones
    B, page, W, n_rows, n_pages = 6, 4, 500, 5000, 900
    lens, t_n, t_table, t_free = ints([0] * B), ints([n_pages]), ints([[-1] * W] * B), ints(range(n_pages))
    buf = torch.empty(B + 1 + 3 * n_rows, dtype=I32, device=DEV)
    cu, *rows = torch.split(buf, [B + 1, n_rows, n_rows, n_rows])
    plan, delta, st = paged.PagePlan(ints([0] * B) if own_lens else lens, cu, *rows, t_n), ints([0] * B), status()
    paged.page_plan(lens, delta, t_table, t_free, t_n, page, n_rows, plan=plan, d_status=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        paged.page_plan(lens, delta, t_table, t_free, t_n, page, n_rows, plan=plan, d_status=st)
    at, table, free = [0] * B, [[-1] * W for _ in range(B)], list(range(n_pages))
    for d in ([1000, 500, 9, 0, 30, 1], [800, 700, 900, 3, 0, -1], [-100, 40, -700, 0, 900, 5], [-10**6] * 3 + [1, 1, 1], [5] * B):
        delta.copy_(ints(d)), st.zero_()
        g.replay()
        slots, want = plan_step(at, d, table, free, page)
        assert int(st) == want and plan.lens.tolist() == at and int(t_n) == len(free)
        assert t_table.tolist() == table and t_free.tolist()[:len(free)] == free
        assert plan.slot.tolist() == slots + [-1] * (n_rows - len(slots)) and int(plan.cu[0]) == 0
        lens.copy_(plan.lens)


def test_plan_in_place_into_a_plan():
    # in_place overwrites lens and n_free: a plan with others is refused, nothing is done
    table, free, lens, n = ints([[-1] * 4] * 2), ints(range(8)), ints([0, 0]), ints([8])
    first = paged.page_plan(lens, ints([5, 0]), table, free, n, 4, 6, in_place=True)
    assert first.lens is lens and first.n_free is n
    other = paged.page_plan(lens, ints([0, 0]), table, free, n, 4, 6)
    for p in (other, paged.PagePlan(lens, other.cu, other.slot, other.row_req, other.row_pos, other.n_free)):
        with pytest.raises(ValueError, match="in_place"):
            paged.page_plan(lens, ints([1, 9]), table, free, n, 4, 6, in_place=True, plan=p)
    assert lens.tolist() == [5, 0] and int(n) == 6
    assert paged.page_plan(lens, ints([1, 2]), table, free, n, 4, 6, in_place=True, plan=first) is first
    assert lens.tolist() == [6, 2] and int(n) == 5 and first.slot.tolist()[:3] == [6 * 4 + 1, 5 * 4, 5 * 4 + 1]


def test_plans_of_two_sizes_at_once():
    # two host threads, each with its own stream: the larger plan's shared memory is not taken away
    lib, calls, bad = paged._lib(), [], []
    for B in (paged.MAX_BATCH, 4000):
        buf, s = torch.zeros(8 * B + 64, dtype=I32, device=DEV), torch.cuda.Stream()
        at = [buf.data_ptr() + 4 * (i * B + 4 * i) for i in range(6)]   # lens, delta, new lens, table, cu, the rest
        args = paged._PLAN.pack(B, 16, 1, 4, 4, at[0], at[1], at[2], at[3], at[5], at[5] + 32, at[5] + 64, at[4], at[5] + 96,
                                at[5] + 128, at[5] + 160)
        calls.append((args, buf, s))
    torch.cuda.synchronize()

    def work(args, s):
        torch.cuda.set_device(DEV)
        for _ in range(4000):
            st = lib.csa2p_page_plan(args, None, s.cuda_stream)
            if st:
                bad.append(st)

    threads = [threading.Thread(target=work, args=(a, s)) for a, _, s in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


# ------------------------------------------------------------------ rotation
def test_rope_strides_apart():
    # every layout whose vectors lie apart, heads between rows and rows between heads among them
    cs, n = cos_sin(50, 16), 0
    for rows, heads, R, H in strides(False):
        x, pos = torch.randn((rows, heads, 16), device=DEV).bfloat16(), torch.arange(rows, device=DEV, dtype=I32)
        out = torch.full((1000,), 5.0, device=DEV).bfloat16().as_strided((rows, heads, 16), (R, H, 1))
        want = turned32(x.float(), pos[None], cs, [8]).bfloat16()
        assert torch.equal(paged.rope_axes(x, pos, cs, out=out), want), (rows, heads, R, H)
        out.copy_(x)
        assert torch.equal(paged.rope_axes(out, pos, cs, out=out), want), (rows, heads, R, H)
        n += 1
    assert n > 100


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


def test_layer_step_without_new_rows():
    # drafts taken back and a request ended, nothing new: a step all the same
    d, cs = 128, cos_sin(100, 32)
    cache = paged.PagedCache.new(8, 16, d)
    state = layers.PagedState(ints([0, 0]), ints([[-1] * 4] * 2), ints(range(8)), ints([8]))
    for T, delta in ((50, [20, 30]), (0, [-5, -30]), (1, [1, 0])):
        x, q, st = torch.randn((T, d), device=DEV).bfloat16(), torch.randn((T, 4, d), device=DEV).bfloat16(), status()
        r = layers.paged_layer(cache, state, layers.PagedInput(q, x, ints(delta), cs), d_v=d, d_status=st)
        assert r.out.shape == (T, 4, d) and int(st) == 0 and bool(torch.isfinite(r.out).all())
    assert state.lens.tolist() == [16, 0] and int(state.n_free) == 7


# ------------------------------------------------------------------ rows that no query sees
@pytest.mark.parametrize("H,page,start,pos0,ratio", [
    (1, 16, 100, None, 1), (16, 1, 101, None, 1), (64, 1, 37, [0], 1), (3, 4, 60, [5], 1), (2, 8, 90, [0], 2), (1, 16, 1000, None, 1)])
def test_attn_leading_pages_given_up(H, page, start, pos0, ratio):
    # a chunk from before kv_start: the pages in front of it are gone, and nobody asks for them
    c = AttnCase([200], [200], H, 128, 128, paged.MXFP4, page, 0, ratio, pos0, [start], seed=24)
    c.table[0, :start // page] = -1
    check(c)


@pytest.mark.parametrize("lens,pos0,window,start,flagged", [
    (320, [400], 5, None, False),        # windows past all the rows held
    (320, [300], 0, [400], False),       # kv_start past them
    (320, [316], 3, None, True), (320, [303], 5, None, True), (320, [300], 5, None, False), (320, [301], 5, None, True),
    (320, [321], 5, None, True), (320, [324], 5, None, False), (310, [300], 0, [306], False), (310, [303], 0, [306], True)])
def test_attn_rows_past_the_table_that_none_sees(lens, pos0, window, start, flagged):
    # the table reaches 304 rows: rows past it are flagged where a query would see them, and only there
    c = AttnCase([304], [4], 16, 128, 128, paged.MXFP4, 16, window, 1, pos0, start, seed=25)
    c.table, c.lens = c.table[:, :19], [lens]
    seen = [range(max(start[0] if start else 0, p + 1 - window if window else 0), min(lens, p + 1)) for p in range(pos0[0], pos0[0] + 4)]
    assert flagged == any(r.stop > 304 and len(r) for r in seen)
    st = status()
    out, lse = c.run(st)
    assert int(st) == (csa2.DEV_BAD_INDEX if flagged else 0)
    empty = torch.tensor([r.start >= min(r.stop, 304) for r in seen], device=DEV)
    assert torch.equal((lse == -math.inf).all(1), empty) and bool((out[empty] == 0).all())


# ------------------------------------------------------------------ values that are not finite, scales far out
def same(got, want):
    """Equal bits, or NaN on both sides."""
    nan = torch.isnan(want)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("d", [32, 576])
@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.NVFP4_E4M3_16, paged.MXFP8])
def test_read_every_scale_byte(fmt, d):
    # row r has scale byte r (and its neighbour in the next block) under random codes, NaN codes among them
    g = torch.Generator(device=DEV).manual_seed(fmt)
    c = paged.PagedCache.new(32, 8, d, fmt)
    c.codes.copy_(torch.randint(0, 256, c.codes.shape, generator=g, device=DEV))
    byte = torch.arange(256, device=DEV).view(32, 8, 1) + torch.arange(c.scales.shape[2], device=DEV) % 2
    c.scales.copy_(byte % 256)
    st = status()
    out = paged.paged_read(c, ints(range(256)), d_status=st)
    assert same(out, values64(c.codes.flatten(0, 1), c.scales.flatten(0, 1), fmt).bfloat16()) and int(st) == 0


def test_read_bf16_as_it_is():
    c = paged.PagedCache.new(65536 // 64, 2, 32, paged.BF16)
    bits = torch.arange(65536, device=DEV, dtype=I32).to(torch.int16)
    c.codes.view(torch.int16).copy_(bits.view(c.codes.shape))
    out = paged.paged_read(c, ints(range(2048)))
    assert torch.equal(out.view(torch.int16).flatten(), bits)


@pytest.mark.parametrize("fmt", [paged.MXFP4, paged.NVFP4_E4M3_16, paged.MXFP8])
@pytest.mark.parametrize("rope", [0, 64])
def test_write_blocks_not_finite(fmt, rope):
    # the block itself, not only those beside it, as the contiguous codecs write it
    g = torch.Generator(device=DEV).manual_seed(fmt + rope)
    x = torch.randn((64, 576), generator=g, device=DEV).bfloat16()
    for r, (col, v) in enumerate([(5, math.inf), (5, -math.inf), (40, math.nan), (511, math.inf), (100, math.nan)]):
        x[r, col] = v
    x[5, 64:96], x[6, 96:112], x[7, :] = math.nan, math.inf, -math.inf
    x[8, 3], x[8, 4] = math.nan, math.inf
    if rope:
        x[9, 520], x[10, 575], x[11, 544:] = math.inf, math.nan, -math.inf
    cs, pos = cos_sin(64, rope) if rope else None, torch.arange(64, device=DEV, dtype=I32)
    c, st = paged.PagedCache.new(4, 16, 576, fmt), status()
    paged.paged_write(c, x, ints(range(64)), *((pos, cs) if rope else ()), d_status=st)
    assert int(st) == csa2.DEV_NONFINITE
    if fmt == paged.MXFP8:
        codes, scales = csa2.quant_fp8(turned32(x.float(), pos[None], cs, [32]) if rope else x)
    elif rope:
        codes, scales = torch.empty_like(c.codes.view(64, -1)), torch.empty_like(c.scales.view(64, -1))
        csa2.csa2_rope_quant_fp4([(x, codes, scales, 64, pos, cs, fmt)])
    else:
        codes, scales = csa2.quant_fp4(x, fmt=fmt)
    assert torch.equal(c.codes.view(64, -1), codes) and torch.equal(c.scales.view(64, -1), scales)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("channels", [[3], [300], [512], [575], [530, 40], [545]])
def test_attn_not_finite_channels(fmt, channels):
    # in rows of 576: each part of a row's staging marks its key, in every tile, for the queries that see it
    c = AttnCase([300, 140, 513], [5, 40, 1], 16, 576, 512, fmt, 16, seed=26)
    for b, j in ((0, 299), (0, 300), (1, 120), (1, 139), (2, 513)):        # 300 and 513 lie past the rows held
        pg, off = int(c.table[b, j // 16]), j % 16
        for ch in channels:
            if fmt == paged.BF16:
                c.cache.codes[pg, off, ch] = math.nan if j % 2 else -math.inf
            elif fmt == paged.MXFP8 and j % 2:
                c.cache.codes[pg, off, ch] = 0x7F
            else:
                c.cache.scales[pg, off, ch // (16 if fmt == paged.NVFP4_E4M3_16 else 32)] = 0xFF
    out, _ = check(c)
    assert int(torch.isnan(out).any(-1).any(-1).sum()) == 1 + 20


# ------------------------------------------------------------------ many requests, far slots
def test_attn_most_requests():
    # 16,384 requests, most without a token: as a call of those that have some
    B, H, d = paged.MAX_BATCH, 2, 64
    r = np.random.default_rng(7)
    new = np.where(r.random(B) < 0.03, r.integers(1, 4, B), 0)
    new[[0, B - 1]] = 2
    lens = new + r.integers(0, 90, B)
    some = new > 0
    table = r.integers(0, 50, (B, 6))
    cache = paged.PagedCache.new(50, 16, d, paged.MXFP8)
    g = torch.Generator(device=DEV).manual_seed(8)
    cache.codes.copy_(torch.randint(0, 0x78, cache.codes.shape, generator=g, device=DEV))
    cache.scales.fill_(120)
    q = torch.randn((int(new.sum()), H, d), generator=g, device=DEV).bfloat16()
    got = []
    for keep in (np.ones(B, bool), some):
        cu, st = np.concatenate([[0], np.cumsum(new[keep])]), status()
        got.append(paged.paged_attn(q, cache, ints(table[keep]), ints(lens[keep]), ints(cu), d_status=st))
        assert int(st) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_plan_most_requests():
    B, page = paged.MAX_BATCH, 4
    r = np.random.default_rng(9)
    steps = [r.integers(0, 9, B), np.where(r.random(B) < 0.5, -r.integers(0, 9, B), 1), np.full(B, -9)]
    lens, run = np.zeros(B, int), []
    for d in steps:
        run.append([int(v) for v in np.maximum(d, -lens)])
        lens = lens + run[-1]
    run_plan(run, [0] * B, [[-1] * 4 for _ in range(B)], list(range(20000)), 20000, page, 80000, True)


@pytest.mark.parametrize("fmt", [paged.BF16, paged.MXFP8])
def test_write_and_read_far_slots(fmt):
    # rows whose byte offsets pass 32 bits
    page, d = 64, 576
    n = (5 << 30) // (page * d * (2 if fmt == paged.BF16 else 1))
    shape = (n, page, d)
    codes = torch.empty(shape, dtype=torch.bfloat16 if fmt == paged.BF16 else torch.uint8, device=DEV)
    c = paged.PagedCache(codes, None if fmt == paged.BF16 else torch.empty((n, page, d // 32), dtype=torch.uint8, device=DEV))
    x = torch.randn((100, d), device=DEV).bfloat16()
    slot = torch.cat([torch.arange(50, device=DEV), n * page - 1 - torch.arange(50, device=DEV)]).to(I32)
    paged.paged_write(c, x, slot)
    out = paged.paged_read(c, slot)
    if fmt == paged.BF16:
        assert torch.equal(out, x) and torch.equal(codes.view(-1, d)[slot.long()], x)
    else:
        want, scales = csa2.quant_fp8(x)
        assert torch.equal(codes.view(-1, d)[slot.long()], want)
        assert torch.equal(out, values64(want, scales, fmt).bfloat16())


# ------------------------------------------------------------------ together
def test_further_layers_of_a_step():
    # two layers of one step share the plan: the second as if it had been first, on its own cache and input
    H, d, fmt = 8, 128, paged.NVFP4_E4M3_16
    g, cs = torch.Generator(device=DEV).manual_seed(27), cos_sin(200, 32)
    new_state = lambda: layers.PagedState(ints([0, 0, 0]), ints([[-1] * 8] * 3), ints(range(20)), ints([20]))  # noqa: E731
    shared, alone = new_state(), new_state()
    caches = [paged.PagedCache.new(20, 16, d, fmt) for _ in range(3)]
    for delta in ([40, 1, 0], [1, 1, 30], [1, -1, 1]):
        T = sum(max(v, 0) for v in delta) + 2
        xs = [layers.PagedInput(torch.randn((T, H, d), generator=g, device=DEV).bfloat16(),
                                torch.randn((T, d), generator=g, device=DEV).bfloat16(), ints(delta), cs) for _ in range(2)]
        st, n = status(), T - 2
        first = layers.paged_layer(caches[0], shared, xs[0], d_v=d, d_status=st)
        again = layers.paged_layer_again(caches[1], shared, xs[1], first.plan, window=20, d_v=d, d_status=st)
        want = layers.paged_layer(caches[2], alone, xs[1], window=20, d_v=d, d_status=st)
        assert int(st) == 0 and again.plan is first.plan
        assert torch.equal(again.out[:n], want.out[:n]) and torch.equal(again.lse[:n], want.lse[:n])
        assert torch.equal(caches[1].codes, caches[2].codes) and torch.equal(caches[1].scales, caches[2].scales)
        assert not torch.equal(caches[0].codes, caches[1].codes)


def test_layer_captured_and_replayed():
    # one captured step of plan, rotation, write and attention, replayed with new rows, as the same steps made one by one
    H, d, B, T = 16, 128, 5, 12
    g, cs = torch.Generator(device=DEV).manual_seed(28), cos_sin(300, 32)
    make = lambda: (paged.PagedCache.new(30, 16, d, paged.MXFP4),                              # noqa: E731
                    layers.PagedState(ints([0] * B), ints([[-1] * 10] * B), ints(range(30)), ints([30])))
    (cache, state), (cache2, state2) = make(), make()
    x = layers.PagedInput(torch.zeros((T, H, d), device=DEV).bfloat16(), torch.zeros((T, d), device=DEV).bfloat16(), ints([0] * B), cs)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layers.paged_layer(cache, state, x, d_v=d)                        # nothing new: only to have run once
    torch.cuda.synchronize()
    graph, st = torch.cuda.CUDAGraph(), status()
    with torch.cuda.graph(graph):
        r = layers.paged_layer(cache, state, x, d_v=d, d_status=st)
    for delta in ([3, 0, 1, 7, 1], [1, 1, 1, 1, 1], [-2, 5, 0, -100, 4], [0, 0, 0, 0, 0], [1, 1, 1, 9, 0]):
        x.q.normal_(generator=g), x.x.normal_(generator=g), x.delta.copy_(ints(delta))
        graph.replay()
        want = layers.paged_layer(cache2, state2, x, d_v=d)
        n = sum(max(v, 0) for v in delta)
        assert torch.equal(r.out[:n], want.out[:n]) and torch.equal(r.lse[:n], want.lse[:n])
        for a, b in ((state.lens, state2.lens), (state.block_table, state2.block_table), (state.n_free, state2.n_free),
                     (r.plan.slot, want.plan.slot), (cache.codes, cache2.codes), (cache.scales, cache2.scales)):
            assert torch.equal(a, b)
    assert int(st) == 0


def test_calls_at_once_on_streams_and_in_graphs():
    # long calls back to back on two streams, then two graphs with workspaces of their own replayed side by side
    cs = [AttnCase([9000, 500], [40, 30], 64, 576, 512, paged.MXFP4, 64, seed=s) for s in (31, 32)]
    args, want, outs, spaces = [], [], [], []
    for c in cs:
        want.append(c.run())
        args.append((c.q, c.cache, torch.from_numpy(c.table).to(DEV).to(I32), ints(c.lens), ints(c.cu)))
        outs.append([(torch.empty_like(want[-1][0]), torch.empty_like(want[-1][1])) for _ in range(6)])
        spaces.append(torch.empty(1 << 27, dtype=torch.uint8, device=DEV))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def calls(i, stream=None):
        for out, lse in outs[i]:
            paged.paged_attn(*args[i], d_v=512, sm_scale=cs[i].sm, out=out, lse=lse, workspace=spaces[i], stream=stream)

    def compare():
        torch.cuda.synchronize()
        for i in range(2):
            for out, lse in outs[i]:
                assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
                out.zero_(), lse.zero_()
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    for i in range(2):
        calls(i, streams[i])
    compare()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            calls(i)
    for _ in range(2):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        compare()
