"""The paged-cache operators as workloads: what is computed, on which inputs, and how much work it is.

Five operators that a server runs together on one layer's paged cache:

* plan   -- block tables, slot map and free list from the requests' lengths
* rope   -- rotary positions with one or several axes on the queries
* write  -- rotation and quantisation of new rows into their pages, and the rows read back as the
            values that the cache holds (write and read are timed together: the cache holds 4 or 8 bits)
* attn   -- attention of new tokens (one, or a chunk, per request) over the pages

With ``own`` the framework's calls are made; otherwise plain 32-bit torch computes the same.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
GROUP = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32, "bf16": 0}      # values of a row that share a scale


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's bookkeeping: every request grows by one row
        {"name": "plan_decode", "op": "plan", "batch": 512, "page": 64, "max_len": 65536, "max_new": 1, "rows": 512, "drop": 0, "mix": 1},
        # a mixed step: chunks, single rows, drafts taken back and requests that end
        {"name": "plan_mixed", "op": "plan", "batch": 193, "page": 64, "max_len": 131072, "max_new": 4096, "rows": 65536, "drop": 30, "mix": 2},
        # queries of one decode step: 32 tokens of text
        {"name": "rope_decode", "op": "rope", "rows": 32, "heads": 64, "d": 576, "rope": 64, "axes": 1, "mix": 3},
        # queries of a chunk with images: time, height and width
        {"name": "rope_vision", "op": "rope", "rows": 4096, "heads": 64, "d": 576, "rope": 64, "axes": 3, "mix": 4},
        # the decoded tokens' rows, in the report's main-KV format
        {"name": "write_decode", "op": "write", "rows": 32, "d": 576, "rope": 64, "axes": 1, "fmt": "nvfp4", "page": 64, "mix": 5},
        # a long prompt's main-KV rows
        {"name": "write_chunk", "op": "write", "rows": 16384, "d": 576, "rope": 64, "axes": 3, "fmt": "mxfp4", "page": 64, "mix": 6},
        # a chunk's sliding-window rows in FP8, an odd number of them
        {"name": "write_swa", "op": "write", "rows": 4099, "d": 576, "rope": 64, "axes": 1, "fmt": "mxfp8", "page": 128, "mix": 7},
        # one token of one sequence with small heads: latency
        {"name": "attn_tiny", "op": "attn", "batch": 1, "new": 1, "ragged": False, "heads": 16, "d": 128, "dv": 128, "max_len": 4096, "ctx": 1.0,
         "fmt": "mxfp4", "page": 64, "window": 0, "ratio": 1, "mix": 8},
        # a decode batch over long sequences of unlike lengths
        {"name": "attn_decode", "op": "attn", "batch": 32, "new": 1, "ragged": False, "heads": 64, "d": 576, "dv": 512, "max_len": 65536, "ctx": 0.5,
         "fmt": "mxfp4", "page": 64, "window": 0, "ratio": 1, "mix": 9},
        # two prompts' chunks of 1,024 tokens, the context already cached
        {"name": "attn_chunk", "op": "attn", "batch": 2, "new": 1024, "ragged": False, "heads": 64, "d": 576, "dv": 512, "max_len": 16384, "ctx": 0.9,
         "fmt": "mxfp4", "page": 64, "window": 0, "ratio": 1, "mix": 10},
        # chunks in a layer that sees its last 128 tokens only, FP8 rows
        {"name": "attn_window", "op": "attn", "batch": 8, "new": 256, "ragged": False, "heads": 64, "d": 576, "dv": 512, "max_len": 2048, "ctx": 0.3,
         "fmt": "mxfp8", "page": 128, "window": 128, "ratio": 1, "mix": 11},
        # decode rows and chunks together, entries that stand for two tokens, small pages
        {"name": "attn_mixed", "op": "attn", "batch": 9, "new": 257, "ragged": True, "heads": 64, "d": 576, "dv": 512, "max_len": 4097, "ctx": 0.1,
         "fmt": "nvfp4", "page": 16, "window": 0, "ratio": 2, "mix": 12},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm, odd ones among them."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "write", "attn", "attn"])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        batch = _spread(rng, 1, 1024)
        new = rng.choice([1, 1, _spread(rng, 2, 4096)])
        return {"op": op, "batch": batch, "page": rng.choice([16, 32, 64, 128]), "max_len": _spread(rng, 64, 131072), "max_new": new,
                "rows": batch if new == 1 else _spread(rng, batch * 2, 65536), "drop": rng.choice([0, 20, 40]), "mix": mix}
    d, dv = rng.choice([(576, 512), (576, 512), (512, 512), (128, 128)])
    rope, axes = rng.choice([32, 64]), rng.choice([1, 2, 3])
    if op == "rope":
        return {"op": op, "rows": _spread(rng, 1, 4096), "heads": rng.choice([8, 16, 32, 64]), "d": d, "rope": rope, "axes": axes, "mix": mix}
    if op == "write":
        return {"op": op, "rows": _spread(rng, 1, 16384), "d": d, "rope": rope, "axes": axes, "fmt": rng.choice(["mxfp4", "nvfp4", "mxfp8", "bf16"]),
                "page": rng.choice([16, 32, 64, 128]), "mix": mix}
    heads = rng.choice([16, 32, 64, 64, 128])
    batch = _spread(rng, 1, 32)
    new = 1 if rng.random() < 0.4 else _spread(rng, 2, 512)
    # padded (request, token, head, key) products and cached rows: no dearer than the listed ones
    most = min(65536, 2_000_000 // batch, 500_000_000 // (batch * new * heads))
    max_len = max(new, _spread(rng, min(64, most), most)) if most > 16 else new
    return {"op": op, "batch": batch, "new": new, "ragged": rng.random() < 0.5, "heads": heads, "d": d, "dv": dv, "max_len": max_len,
            "ctx": rng.choice([0.1, 0.5, 0.9]), "fmt": rng.choice(["mxfp4", "mxfp4", "nvfp4", "mxfp8", "bf16"]), "page": rng.choice([16, 32, 64, 128]),
            "window": rng.choice([0, 0, 128, 1000]), "ratio": rng.choice([1, 1, 2]), "mix": mix}


def _lengths(c):
    """Lengths of an attention case, from the case alone: (cached entries, new tokens) of each request."""
    r = random.Random(c["mix"])
    new = [r.randint(0, c["new"]) if c["ragged"] and i else c["new"] for i in range(c["batch"])]
    lens = [max(-(-n // c["ratio"]), r.randint(int(c["ctx"] * c["max_len"]), c["max_len"])) if i else c["max_len"] for i, n in enumerate(new)]
    return lens, new


def _steps(c):
    """Lengths before a plan case's step and their changes, from the case alone."""
    r = random.Random(c["mix"])
    old = [r.randint(0, c["max_len"]) for _ in range(c["batch"])]
    left, delta = c["rows"], []
    for i in range(c["batch"]):
        what = r.randrange(100)
        if what < c["drop"]:
            delta.append(-old[i] if what % 2 else -min(old[i], r.randint(1, 4)))     # ended, or drafts taken back
        else:
            n = min(left, 1 if r.random() < 0.5 else r.randint(1, c["max_new"]))
            delta.append(n)
            left -= n
    return old, delta


def _row_bytes(c):
    g = GROUP[c["fmt"]]
    return {"mxfp4": c["d"] // 2, "nvfp4": c["d"] // 2, "mxfp8": c["d"], "bf16": 2 * c["d"]}[c["fmt"]] + (c["d"] // g if g else 0)


def work(c):
    if c["op"] == "plan":
        old, delta = _steps(c)
        n = sum(max(0, d) for d in delta)
        pages = sum(abs(-(-(o + d) // c["page"]) - -(-o // c["page"])) for o, d in zip(old, delta))
        return {"bytes": 16 * c["batch"] + 12 * c["rows"] + 8 * pages, "flops": n}
    if c["op"] == "rope":
        return {"bytes": c["rows"] * (4 * c["heads"] * c["d"] + 4 * c["axes"]), "flops": 3 * c["rows"] * c["heads"] * c["rope"]}
    if c["op"] == "write":
        return {"bytes": c["rows"] * (2 * c["d"] + 2 * _row_bytes(c) + 2 * c["d"] + 4 * c["axes"] + 4), "flops": 6 * c["rows"] * c["d"]}
    pairs = rows = 0
    lens, new = _lengths(c)
    for n, t in zip(lens, new):
        p = n * c["ratio"] - t + np.arange(t) + 1
        hi = np.minimum(n, p // c["ratio"])
        lo = np.maximum(0, p // c["ratio"] - c["window"]) if c["window"] else np.zeros_like(hi)
        pairs += int(np.maximum(0, hi - lo).sum())
        rows += int(max(0, hi.max() - lo.min())) if t else 0
    pairs *= c["heads"]
    tokens = sum(new)
    return {"bytes": rows * (_row_bytes(c) + 4 / c["page"]) + tokens * c["heads"] * (2 * c["d"] + 2 * c["dv"] + 4),
            "flops": 2 * pairs * (c["d"] + c["dv"])}


# ------------------------------------------------------------------------------------------ inputs
def _table(rope, n_pos):
    """Cosines, then sines, of position x base^(-2i / rope); the angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rope, 2, device=DEV, dtype=torch.float64) / rope)
    a = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _sections(rope, axes):
    """Pairs that each axis turns: equal parts, the first takes what is left over."""
    n = rope // 2 // axes
    return [rope // 2 - n * (axes - 1)] + [n] * (axes - 1)


def _positions(g, rows, axes):
    """Text: one running position. Images: the frame's, and the patch's row and column."""
    t = torch.arange(rows, device=DEV) + torch.randint(0, 60000, (1,), generator=g, device=DEV)
    if axes == 1:
        return t.int()
    grid = [t // 1024, t // 32 % 32, t % 32]
    return torch.stack(grid[:axes]).int()


def _latents(g, n, d):
    """Rows as a layer makes them: normal values, channels of unlike size."""
    x = torch.randn((n, d), generator=g, device=DEV)
    return (x * torch.exp2(torch.randn((d,), generator=g, device=DEV) * 0.5)).bfloat16()


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + c["mix"])
    s = dict(c)
    if c["op"] == "plan":
        old, delta = _steps(c)
        width = -(-(c["max_len"] + c["max_new"]) // c["page"])
        held = [-(-o // c["page"]) for o in old]
        n_pages = sum(held) + sum(-(-d // c["page"]) + 1 for d in delta if d > 0) + 64
        order = torch.randperm(n_pages, generator=g, device=DEV).int()
        held_t = torch.tensor(held, device=DEV)
        j = torch.arange(width, device=DEV)
        first = held_t.cumsum(0) - held_t
        table = torch.where(j < held_t[:, None], order[(first[:, None] + j).clamp(max=n_pages - 1)], -1).int()
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
        n = n_pages - sum(held)
        free[:n] = order[sum(held):]
        s.update(lens=torch.tensor(old, dtype=torch.int32, device=DEV), delta=torch.tensor(delta, dtype=torch.int32, device=DEV), table=table,
                 free=free, n_free=torch.tensor([n], dtype=torch.int32, device=DEV))
    elif c["op"] == "rope":
        s.update(x=torch.randn((c["rows"], c["heads"], c["d"]), generator=g, device=DEV).bfloat16(), pos=_positions(g, c["rows"], c["axes"]),
                 cs=_table(c["rope"], 65536), sections=_sections(c["rope"], c["axes"]))
    elif c["op"] == "write":
        pages = -(-c["rows"] // c["page"]) + 7
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * c["page"] + torch.arange(c["page"], device=DEV)
        codes, scales = _empty(c, pages)
        s.update(x=_latents(g, c["rows"], c["d"]), slot=slots.reshape(-1)[3:3 + c["rows"]].int(), codes=codes, scales=scales,
                 pos=_positions(g, c["rows"], c["axes"]), cs=_table(c["rope"], 80000), sections=_sections(c["rope"], c["axes"]))
    else:
        lens, new = _lengths(c)
        need = [-(-n // c["page"]) for n in lens]
        width, pages = max(need) + 1, sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).int()
        first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
        j = torch.arange(width, device=DEV)
        table = torch.where(j < torch.tensor(need, device=DEV)[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], -1).int()
        parts = [_quant(_latents(g, min(1 << 18, pages * c["page"] - at), c["d"]).float(), c["fmt"]) for at in range(0, pages * c["page"], 1 << 18)]
        codes = torch.cat([p[0] for p in parts]).view(pages, c["page"], -1)
        scales = torch.cat([p[1] for p in parts]).view(pages, c["page"], -1) if GROUP[c["fmt"]] else None
        cu = torch.tensor([0] + new, device=DEV).cumsum(0).int()
        lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s.update(q=torch.randn((sum(new), c["heads"], c["d"]), generator=g, device=DEV).bfloat16(), table=table, lens=lens, cu=cu, codes=codes,
                 scales=scales, pos0=lens * c["ratio"] - (cu[1:] - cu[:-1]), scale=1.0 / math.sqrt(c["d"]), max_new=max(new))
    return s


# ------------------------------------------------------------------------------------------ formats
def _empty(c, pages):
    rows = (pages, c["page"])
    if c["fmt"] == "bf16":
        return torch.zeros(rows + (c["d"],), dtype=torch.bfloat16, device=DEV), None
    width = c["d"] if c["fmt"] == "mxfp8" else c["d"] // 2
    return torch.zeros(rows + (width,), dtype=torch.uint8, device=DEV), torch.zeros(rows + (c["d"] // GROUP[c["fmt"]],), dtype=torch.uint8, device=DEV)


def _power(byte):
    """2^(byte - 127) in 32 bits."""
    b = byte.int()
    return torch.where(b > 0, b << 23, 1 << 22).int().view(torch.float32)


def _quant(x, fmt):
    """Rows of 32-bit values as codes and scale bytes."""
    if fmt == "bf16":
        return x.bfloat16(), None
    b = x.view(x.shape[0], -1, GROUP[fmt])
    top = b.abs().amax(2)
    if fmt == "nvfp4":
        sc = (top / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        v, scales = b / sc.float()[..., None], sc.view(torch.uint8)
    else:
        e = (torch.frexp(top).exponent - 1 - (2 if fmt == "mxfp4" else 8)).clamp(-127, 127)
        scales = (torch.where(top > 0, e, 0) + 127).to(torch.uint8)
        v = b / _power(scales)[..., None]
    if fmt == "mxfp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape), scales
    a = v.abs()
    code = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(b)).view(x.shape)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scales


def _values(codes, scales, fmt):
    """The 32-bit values of rows [..., bytes] of codes and their scale bytes."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
        pair = torch.stack([lut[torch.arange(256, device=DEV) % 16], lut[torch.arange(256, device=DEV) // 16]], 1)
        v = pair[codes.int()].flatten(-2)
    sc = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _power(scales)
    return (v.unflatten(-1, (-1, GROUP[fmt])) * sc[..., None]).flatten(-2)


def _rotated(x, s):
    """32-bit rows [..., d] with their last channels turned, pair by pair; one rounding for each product and sum."""
    half = s["rope"] // 2
    pos = s["pos"].view(-1, s["pos"].shape[-1]).long()
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEV), torch.tensor(s["sections"], device=DEV), output_size=half)
    at, i = pos[axis].T, torch.arange(half, device=DEV)
    c, n = s["cs"][at, i], s["cs"][at, half + i]
    c, n = (t.view((t.shape[0],) + (1,) * (x.dim() - 2) + (half,)) for t in (c, n))
    a, b = x[..., -s["rope"]::2], x[..., 1 - s["rope"]::2]
    turned = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    return torch.cat([x[..., :-s["rope"]], turned], -1)


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else {"plan": _plan, "rope": _rope, "write": _write, "attn": _attn}[s["op"]](s)


def _own(s):
    from fp4_kv_cache_gb300 import paged

    if s["op"] == "plan":
        p = paged.page_plan(s["lens"], s["delta"], s["table"], s["free"], s["n_free"], s["page"], s["rows"])
        return [p.lens, p.cu, p.slot, p.row_req, p.row_pos, p.n_free, s["table"], s["free"]]
    if s["op"] == "rope":
        return paged.rope_axes(s["x"], s["pos"], s["cs"], s["sections"])
    cache = paged.PagedCache(s["codes"], s["scales"])
    if s["op"] == "write":
        paged.paged_write(cache, s["x"], s["slot"], s["pos"], s["cs"], s["sections"])
        return paged.paged_read(cache, s["slot"])
    return paged.paged_attn(s["q"], cache, s["table"], s["lens"], s["cu"], s["pos0"], d_v=s["dv"], window=s["window"], ratio_m=s["ratio"],
                            sm_scale=s["scale"])


def _plan(s):
    page, table, free = s["page"], s["table"], s["free"]
    old, n0 = s["lens"].long(), s["n_free"].long()
    lens = (old + s["delta"]).clamp(min=0)
    had, has = (old + page - 1) // page, (lens + page - 1) // page
    j = torch.arange(table.shape[1], device=DEV)
    back, take = (had - has).clamp(min=0), (has - had).clamp(min=0)
    # pages given back go on top of the free list, in order; pages taken come from its top
    gone = (j >= has[:, None]) & (j < had[:, None])
    at = torch.where(gone, n0 + (back.cumsum(0) - back)[:, None] + j - has[:, None], free.shape[0])
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at.reshape(-1), table.reshape(-1))
    top = n0 + back.sum()
    want = (j >= had[:, None]) & (j < has[:, None])
    at = top - 1 - (take.cumsum(0) - take)[:, None] - (j - had[:, None])
    table.copy_(torch.where(want, torch.where(at >= 0, stack[at.clamp(0, free.shape[0] - 1)], -1), table))
    n_free = (top - take.sum()).clamp(min=0)
    free.copy_(torch.where(torch.arange(free.shape[0], device=DEV) < n_free, stack[:-1], free))
    new = (lens - old).clamp(min=0)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    r = torch.arange(s["rows"], device=DEV)
    req = torch.searchsorted(cu[1:], r, right=True)
    real = req < old.shape[0]
    req = req.clamp(max=old.shape[0] - 1)
    pos = old[req] + r - cu[req]
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return [lens.int(), cu.int()] + [torch.where(real, v, -1).int() for v in (slot, req, pos)] + [n_free.int(), table, free]


def _rope(s):
    return _rotated(s["x"].float(), s).bfloat16()


def _write(s):
    codes, scales = _quant(_rotated(s["x"].float(), s), s["fmt"])
    at = s["slot"].long()
    s["codes"].flatten(0, 1)[at] = codes
    if scales is None:
        return s["codes"].flatten(0, 1)[at]
    s["scales"].flatten(0, 1)[at] = scales
    return _values(s["codes"].flatten(0, 1)[at], s["scales"].flatten(0, 1)[at], s["fmt"]).bfloat16()


def _attn(s):
    page, heads, most = s["page"], s["heads"], s["max_new"]
    t = s["table"].clamp(min=0)
    k = _values(s["codes"][t], s["scales"][t] if s["scales"] is not None else None, s["fmt"]).flatten(1, 2)
    n, cu = s["lens"].long(), s["cu"].long()
    # requests padded to the longest chunk: [request, token x head, channel]
    i = torch.arange(most, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].flatten(1, 2)
    seen = (s["pos0"].long()[:, None] + i + 1).clamp(min=0) // s["ratio"]
    j = torch.arange(k.shape[1], device=DEV)
    see = (j < torch.minimum(seen, n[:, None])[..., None])
    if s["window"]:
        see &= j >= (seen - s["window"])[..., None]
    logit = (q @ k.mT * s["scale"]).unflatten(1, (most, heads)).masked_fill_(~see[:, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = logit.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1)
    o = (p.flatten(1, 2) @ k[..., :s["dv"]]).unflatten(1, (most, heads)) / torch.where(total > 0, total, 1.0)[..., None]
    lse = top[..., 0] + total.log()
    r = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], r, right=True)
    return o[b, r - cu[b]].bfloat16(), torch.where(total > 0, lse, -math.inf)[b, r - cu[b]]


# ------------------------------------------------------------------------------------------ 64 bits
def _decode64(codes, scales, fmt):
    """Values of rows of codes in 64 bits, bit field by bit field."""
    if fmt == "bf16":
        return codes.double()
    if fmt == "mxfp8":
        b = codes.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(e > 0, (8 + m) * _power64(e - 10), m * 2.0 ** -9) * (1.0 - 2.0 * (b >> 7))
    else:
        b = torch.stack([codes.long() & 15, codes.long() >> 4], -1).flatten(-2)
        e, m = (b >> 1) & 3, (b & 1).double()
        v = torch.where(e > 0, (2 + m) * _power64(e - 2), m / 2) * (1.0 - 2.0 * (b >> 3))
    sb = scales.long()
    if fmt == "nvfp4":
        e, m = (sb >> 3) & 15, (sb & 7).double()
        sc = torch.where(e > 0, (8 + m) * _power64(e - 10), m * 2.0 ** -9)
    else:
        sc = _power64(sb - 127)
    return v * sc.repeat_interleave(GROUP[fmt], -1)


def _turn64(x, s):
    """The rotation in 64 bits, channel by channel: even channels a c - b n, odd ones a n + b c; products and sums rounded to 32 bits
    where `x` is a cache row, as the cache's definition has it (64-bit products of these values are exact)."""
    d, rope = x.shape[-1], s["rope"]
    y = x.clone()
    pos = s["pos"].reshape(len(s["sections"]), -1).long()
    bounds = np.cumsum(s["sections"])
    r32 = (lambda v: v.float().double()) if s["op"] == "write" else (lambda v: v)
    for i in range(rope // 2):
        at = pos[int(np.searchsorted(bounds, i, side="right"))]
        c, n = s["cs"][at, i].double(), s["cs"][at, rope // 2 + i].double()
        a, b = x[..., d - rope + 2 * i], x[..., d - rope + 2 * i + 1]
        if a.dim() == 2:
            c, n = c[:, None], n[:, None]
        y[..., d - rope + 2 * i] = r32(r32(a * c) - r32(b * n))
        y[..., d - rope + 2 * i + 1] = r32(r32(a * n) + r32(b * c))
    return y


def _power64(e):
    """2^e in 64 bits for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest64(v, grid):
    """Values of `grid` nearest to v >= 0, ties to the even place."""
    grid = torch.tensor(grid, dtype=torch.float64, device=DEV)
    hi = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
    lo = hi - 1
    up = (grid[hi] - v < v - grid[lo]) | ((grid[hi] - v == v - grid[lo]) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def exact(c, seed):
    if c["op"] == "plan":
        return None                                     # whole numbers
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _turn64(s["x"].double(), s)
    if c["op"] == "write":
        y = _turn64(s["x"].double(), s)
        if c["fmt"] == "bf16":
            return y
        b = y.unflatten(-1, (-1, GROUP[c["fmt"]]))
        top = b.abs().amax(-1, keepdim=True)
        e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
        if c["fmt"] == "nvfp4":
            sc = _nearest64((top / 6).clamp(max=448.0), e4m3)
        else:
            sc = _power64(((top.view(torch.int64) >> 52) - 1023 - (2 if c["fmt"] == "mxfp4" else 8)).clamp(-127, 127))
        grid = e4m3 if c["fmt"] == "mxfp8" else [0, .5, 1, 1.5, 2, 3, 4, 6]
        v = _nearest64((b.abs() / sc).clamp(max=grid[-1]), grid)
        return (v * sc * torch.where(b < 0, -1.0, 1.0)).flatten(-2)
    lens, new = _lengths(c)
    out = torch.zeros((sum(new), c["heads"], c["dv"]), dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b, (n, t) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-n // c["page"])].long()
        k = _decode64(s["codes"][pages].flatten(0, 1)[:n], s["scales"][pages].flatten(0, 1)[:n] if s["scales"] is not None else None, c["fmt"])
        for at in range(0, t, 64):                      # 64 tokens at a time
            m = min(64, t - at)
            q = s["q"][first + at:first + at + m].double()
            last = (n * c["ratio"] - t + at + torch.arange(m, device=DEV) + 1).div(c["ratio"], rounding_mode="floor")
            j = torch.arange(n, device=DEV)
            see = (j < last[:, None]) & ((j >= last[:, None] - c["window"]) | (c["window"] == 0))
            z = (q.flatten(0, 1) @ k.T * s["scale"]).view(m, c["heads"], n).masked_fill(~see[:, None], -math.inf)
            lse[first + at:first + at + m] = torch.logsumexp(z, -1)
            w = torch.exp(z - lse[first + at:first + at + m].clamp(min=-1e300)[..., None])
            out[first + at:first + at + m] = (w.flatten(0, 1) @ k[:, :c["dv"]]).view(m, c["heads"], -1)
        first += t
    return out, lse
