"""Drafted tokens and shared pages over the paged cache, as workloads: what is computed, on which
inputs, and how much work it is.

Three operators that a server runs on the paged cache beside plan, write and attention:

* tree   -- attention of a tree of drafted tokens over the pages (the tree's positions and its mask,
            then the attention)
* verify -- which drafted tokens stay, by the target's probabilities and given random numbers, and the
            token that follows them
* pages  -- rows of the drafts that stay moved together (compact); requests that share a prompt's pages:
            forked, their last pages copied, and ended again (fork)

With ``own`` the framework's calls are made; otherwise plain torch computes the same: attention in 32
bits, whole numbers in 64.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
GROUP = {"mxfp4": 32, "nvfp4": 16, "mxfp8": 32, "bf16": 0}      # values of a row that share a scale
FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence with small heads and a chain of five drafts behind its last token: latency
        {"name": "tree_one", "op": "tree", "batch": 1, "nodes": 6, "shape": "chain", "ragged": False, "heads": 16, "d": 128, "dv": 128,
         "max_len": 4096, "ctx": 1.0, "fmt": "mxfp4", "page": 64, "window": 0, "mix": 1},
        # a decode batch over long sequences, five drafts each
        {"name": "tree_chain", "op": "tree", "batch": 32, "nodes": 6, "shape": "chain", "ragged": False, "heads": 64, "d": 576, "dv": 512,
         "max_len": 65536, "ctx": 0.5, "fmt": "mxfp4", "page": 64, "window": 0, "mix": 2},
        # few sequences with wide trees, as many nodes as 64 for some and fewer for others
        {"name": "tree_wide", "op": "tree", "batch": 4, "nodes": 64, "shape": "tree", "ragged": True, "heads": 64, "d": 576, "dv": 512,
         "max_len": 16384, "ctx": 0.7, "fmt": "nvfp4", "page": 16, "window": 0, "mix": 3},
        # a layer that sees its last 128 tokens only, FP8 rows
        {"name": "tree_window", "op": "tree", "batch": 16, "nodes": 25, "shape": "tree", "ragged": True, "heads": 64, "d": 576, "dv": 512,
         "max_len": 2048, "ctx": 0.3, "fmt": "mxfp8", "page": 128, "window": 128, "mix": 4},
        # one sequence's five drafts
        {"name": "verify_one", "op": "verify", "batch": 1, "nodes": 6, "shape": "chain", "ragged": False, "vocab": 131072, "dtype": "f32",
         "drafts": "drawn", "near": 0.7, "mix": 5},
        # a batch's trees: drafts drawn from a smaller model's probabilities
        {"name": "verify_batch", "op": "verify", "batch": 64, "nodes": 16, "shape": "tree", "ragged": True, "vocab": 131072, "dtype": "f32",
         "drafts": "drawn", "near": 0.7, "mix": 6},
        # drafts that are certain (looked up in the text so far), probabilities in 16 bits, an odd vocabulary
        {"name": "verify_sure", "op": "verify", "batch": 33, "nodes": 9, "shape": "tree", "ragged": True, "vocab": 32003, "dtype": "bf16",
         "drafts": "sure", "near": 0.5, "mix": 7},
        # a batch's small trees, the four caches that a model's layers share
        {"name": "compact_few", "op": "compact", "batch": 32, "nodes": 6, "caches": 4, "fmts": "mxfp4", "d": 576, "page": 64, "max_len": 4096, "mix": 8},
        # wide trees over small pages, a window layer's FP8 rows among the caches
        {"name": "compact_wide", "op": "compact", "batch": 64, "nodes": 64, "caches": 20, "fmts": "nvfp4+mxfp8", "d": 576, "page": 16, "max_len": 513, "mix": 9},
        # eight answers to one prompt
        {"name": "fork_one", "op": "fork", "prompts": 1, "samples": 8, "caches": 4, "fmts": "mxfp4", "d": 576, "page": 64, "max_len": 32771, "mix": 10},
        # many prompts with 32 answers each
        {"name": "fork_batch", "op": "fork", "prompts": 16, "samples": 32, "caches": 4, "fmts": "mxfp4", "d": 576, "page": 64, "max_len": 65536, "mix": 11},
        # short prompts over small pages, rows of two formats
        {"name": "fork_short", "op": "fork", "prompts": 37, "samples": 3, "caches": 6, "fmts": "bf16+mxfp8", "d": 128, "page": 16, "max_len": 700, "mix": 12},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm, odd ones among them."""
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "compact", "fork"])
    mix = rng.randrange(1 << 20)
    shape = rng.choice(["chain", "tree", "tree"])
    if op == "tree":
        heads, (d, dv) = rng.choice([16, 32, 64, 64, 128]), rng.choice([(576, 512), (576, 512), (512, 512), (128, 128)])
        batch, nodes = _spread(rng, 1, 32), _spread(rng, 1, 128)
        # padded (request, node, head, key) products and cached rows: no dearer than the listed ones
        most = max(nodes, min(65536, 2_000_000 // batch, 400_000_000 // (batch * nodes * heads)))
        return {"op": op, "batch": batch, "nodes": nodes, "shape": shape, "ragged": rng.random() < 0.5, "heads": heads, "d": d, "dv": dv,
                "max_len": max(nodes, _spread(rng, min(64, most), most)), "ctx": rng.choice([0.1, 0.5, 0.9]),
                "fmt": rng.choice(["mxfp4", "mxfp4", "nvfp4", "mxfp8", "bf16"]), "page": rng.choice([16, 32, 64, 128]),
                "window": rng.choice([0, 0, 128, 1000]), "mix": mix}
    if op == "verify":
        nodes = _spread(rng, 1, 32)
        vocab = _spread(rng, 1000, 131072)
        return {"op": op, "batch": _spread(rng, 1, max(1, 130_000_000 // (nodes * vocab)) if nodes * vocab > 2_000_000 else 64), "nodes": nodes,
                "shape": shape, "ragged": rng.random() < 0.5, "vocab": vocab, "dtype": rng.choice(["f32", "f32", "f16", "bf16"]),
                "drafts": rng.choice(["drawn", "drawn", "sure"]), "near": rng.choice([0.3, 0.7, 1.5]), "mix": mix}
    d, page = rng.choice([576, 576, 512, 128]), rng.choice([16, 32, 64, 128])
    fmts = rng.choice(["mxfp4", "nvfp4", "mxfp8", "bf16", "mxfp4+mxfp8", "nvfp4+bf16"])
    if op == "compact":
        nodes = _spread(rng, 1, 64)
        return {"op": op, "batch": _spread(rng, 1, 64), "nodes": nodes, "caches": _spread(rng, 1, 20), "fmts": fmts, "d": d, "page": page,
                "max_len": max(nodes, _spread(rng, 16, 513)), "mix": mix}
    prompts = _spread(rng, 1, 37)
    return {"op": op, "prompts": prompts, "samples": _spread(rng, 1, max(1, 512 // prompts)), "caches": _spread(rng, 1, 6), "fmts": fmts, "d": d,
            "page": page, "max_len": _spread(rng, 16, 200_000 // prompts), "mix": mix}


def _trees(c):
    """Nodes of each request and their parents, from the case alone: node 0 is the last token, the others are drafts, parents first."""
    r = random.Random(c["mix"])
    sizes = [r.randint(1, c["nodes"]) if c["ragged"] and i else c["nodes"] for i in range(c["batch"])]
    return sizes, [[i - 1 if c["shape"] == "chain" or i == 0 else r.randrange(max(0, i - 7), i) for i in range(n)] for n in sizes]


def _lengths(c, sizes):
    """Rows held by each request, the nodes among them."""
    r = random.Random(c["mix"] + 1)
    return [max(n, r.randint(int(c.get("ctx", 0.2) * c["max_len"]), c["max_len"])) if i else c["max_len"] for i, n in enumerate(sizes)]


def _paths(c):
    """A compact case: nodes of each request, and the nodes that stay."""
    r = random.Random(c["mix"])
    sizes = [r.randint(1, c["nodes"]) if i else c["nodes"] for i in range(c["batch"])]
    return sizes, [[0] + sorted(r.sample(range(1, n), r.randint(0, min(n - 1, 7)))) for n in sizes]


def _prompts(c):
    """A fork case: rows of each prompt."""
    r = random.Random(c["mix"])
    return [c["max_len"] if i == 0 else r.randint(c["max_len"] // 8 + 1, c["max_len"]) for i in range(c["prompts"])]


def _row_bytes(d, fmt):
    g = GROUP[fmt]
    return {"mxfp4": d // 2, "nvfp4": d // 2, "mxfp8": d, "bf16": 2 * d}[fmt] + (d // g if g else 0)


def _cache_bytes(c):
    """Bytes of one row in all caches."""
    f = c["fmts"].split("+")
    return sum(_row_bytes(c["d"], f[i % len(f)]) for i in range(c["caches"]))


def work(c):
    if c["op"] == "tree":
        sizes, parents = _trees(c)
        pairs = rows = 0
        for n, size, parent in zip(_lengths(c, sizes), sizes, parents):
            depth = []
            for i, p in enumerate(parent):
                depth.append(0 if p < 0 else depth[p] + 1)
                pairs += depth[i] + 1 if not c["window"] else min(depth[i] + 1, c["window"])
                pairs += n - size if not c["window"] else max(0, min(n - size, c["window"] - depth[i] - 1))
            rows += size + (n - size if not c["window"] else min(n - size, c["window"] - 1))
        pairs *= c["heads"]
        tokens = sum(sizes)
        return {"bytes": rows * (_row_bytes(c["d"], c["fmt"]) + 4 / c["page"]) + tokens * (c["heads"] * (2 * c["d"] + 2 * c["dv"] + 4) + 12),
                "flops": 2 * pairs * (c["d"] + c["dv"])}
    if c["op"] == "verify":
        # each request's last kept node: its row of the target's probabilities, and of the drafts' where they were drawn
        size = FLOAT[c["dtype"]].itemsize
        rows = 2 if c["drafts"] == "drawn" and c["nodes"] > 1 else 1
        return {"bytes": c["batch"] * (rows * c["vocab"] * size + 8) + 12 * sum(_trees(c)[0]), "flops": 2 * c["batch"] * c["vocab"]}
    if c["op"] == "compact":
        moved = sum(sum(i != p for i, p in enumerate(path)) for path in _paths(c)[1])
        return {"bytes": 2 * moved * _cache_bytes(c) + 16 * c["batch"] + 8 * moved, "flops": moved}
    lens = _prompts(c)
    full, part = sum(n // c["page"] for n in lens), sum(n % c["page"] for n in lens)
    # fork: a prompt's table entries read once, written for each answer, its pages counted up; last pages copied; ended: entries read, counted down
    return {"bytes": full * (4 + 8 + 4 * c["samples"]) + part * (1 + c["samples"]) * _cache_bytes(c) + full * (8 + 4 * c["samples"]) + 16 * c["prompts"] * c["samples"],
            "flops": 2 * full * c["samples"]}


# ------------------------------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _latents(g, n, d):
    """Rows as a layer makes them: normal values, channels of unlike size."""
    x = torch.randn((n, d), generator=g, device=DEV)
    return (x * torch.exp2(torch.randn((d,), generator=g, device=DEV) * 0.5)).bfloat16()


def _pages(g, lens, page, spare, extra=1):
    """A block table over pages in random order, and the pages that are not in it."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).int()
    first = torch.tensor(np.cumsum([0] + need[:-1]), device=DEV)
    j = torch.arange(max(need) + extra, device=DEV)
    table = torch.where(j < torch.tensor(need, device=DEV)[:, None], order[(first[:, None] + j).clamp(max=order.shape[0] - 1)], -1).int()
    return table, order[sum(need):]


def _bytes(g, c, pages):
    """Caches of any bytes: (codes, scales) of each."""
    f, made = c["fmts"].split("+"), []
    for i in range(c["caches"]):
        fmt = f[i % len(f)]
        width = {"mxfp4": c["d"] // 2, "nvfp4": c["d"] // 2, "mxfp8": c["d"], "bf16": 2 * c["d"]}[fmt]
        codes = torch.randint(0, 120, (pages, c["page"], width), generator=g, device=DEV, dtype=torch.uint8)
        scales = torch.randint(100, 120, (pages, c["page"], c["d"] // GROUP[fmt]), generator=g, device=DEV, dtype=torch.uint8) if GROUP[fmt] else None
        made.append((codes.view(torch.bfloat16) if fmt == "bf16" else codes, scales))
    return made


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 1000003 + c["mix"])
    s = dict(c)
    if c["op"] in ("tree", "verify"):
        sizes, parents = _trees(c)
        s.update(parent=_ints([p for q in parents for p in q]), cu=_ints(np.cumsum([0] + sizes).tolist()))
    if c["op"] == "tree":
        lens = _lengths(c, sizes)
        table, spare = _pages(g, lens, c["page"], 3)
        rows = (sum(-(-n // c["page"]) for n in lens) + 3) * c["page"]
        parts = [_quant(_latents(g, min(1 << 18, rows - at), c["d"]).float(), c["fmt"]) for at in range(0, rows, 1 << 18)]
        s.update(q=torch.randn((sum(sizes), c["heads"], c["d"]), generator=g, device=DEV).bfloat16(), table=table, lens=_ints(lens),
                 codes=torch.cat([p[0] for p in parts]).view(rows // c["page"], c["page"], -1),
                 scales=torch.cat([p[1] for p in parts]).view(rows // c["page"], c["page"], -1) if GROUP[c["fmt"]] else None,
                 scale=1.0 / math.sqrt(c["d"]))
    elif c["op"] == "verify":
        # a target's logits, most of them far below a few; the smaller model's are near to them; siblings are drawn from their parent's row
        shape = (sum(sizes), c["vocab"])
        logits = torch.randn(shape, generator=g, device=DEV).mul_(2.0)
        logits[:, torch.randint(0, c["vocab"], (40,), generator=g, device=DEV)] += 8.0
        drafted = torch.randn(shape, generator=g, device=DEV).mul_(c["near"]).add_(logits)
        first = torch.tensor(np.repeat(np.cumsum([0] + sizes[:-1]), sizes), device=DEV)
        up = first + s["parent"].long().clamp(min=0)
        token = torch.cat([(drafted[up[at:at + 256]] - torch.empty((min(256, shape[0] - at), shape[1]), device=DEV).exponential_(generator=g).log_()).argmax(1)
                           for at in range(0, shape[0], 256)])
        s.update(p=torch.softmax(logits, 1).to(FLOAT[c["dtype"]]), token=token.int(), u=torch.rand(shape[0], generator=g, device=DEV),
                 r=torch.rand(c["batch"], generator=g, device=DEV), q=torch.softmax(drafted, 1).to(FLOAT[c["dtype"]]) if c["drafts"] == "drawn" else None)
    elif c["op"] == "compact":
        sizes, paths = _paths(c)
        lens = _lengths(c, sizes)
        table, spare = _pages(g, lens, c["page"], 3)
        width = max(len(p) for p in paths)
        s.update(table=table, lens=_ints(lens), cu=_ints(np.cumsum([0] + sizes).tolist()), keep=_ints([len(p) for p in paths]),
                 path=_ints([p + [-1] * (width - len(p)) for p in paths]), data=_bytes(g, c, int(sum(-(-n // c["page"]) for n in lens) + 3)))
    else:
        # prompts in the first places, the answers' places behind them empty
        n = c["prompts"] * c["samples"]
        lens = _prompts(c)
        table, spare = _pages(g, lens + [0] * n, c["page"], n + 5, 3)
        pages = int(sum(-(-v // c["page"]) for v in lens)) + n + 5
        free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        free[:spare.shape[0]] = spare
        source = [-1] * c["prompts"] + [i // c["samples"] for i in range(n)]
        s.update(lens=_ints(lens + [0] * n), table=table, free=free, n_free=_ints([spare.shape[0]]), shares=torch.zeros(pages, dtype=torch.int32, device=DEV),
                 source=_ints(source), ends=_ints([int(v >= 0) for v in source]), data=_bytes(g, c, pages))
    return s


# ------------------------------------------------------------------------------------------ formats
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


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else {"tree": _tree, "verify": _verify, "compact": _compact, "fork": _fork}[s["op"]](s)


def _own(s):
    from fp4_kv_cache_gb300 import draft, paged

    if s["op"] == "tree":
        t = draft.tree_plan(s["parent"], s["lens"], s["cu"], s["nodes"])
        cache = paged.PagedCache(s["codes"], s["scales"])
        out, lse = draft.tree_attn(s["q"], cache, s["table"], s["lens"], s["cu"], t.seen, t.pos, d_v=s["dv"], window=s["window"], sm_scale=s["scale"])
        return t.pos, t.seen, out, lse
    if s["op"] == "verify":
        v = draft.tree_verify(s["p"], s["token"], s["parent"], s["cu"], s["u"], s["r"], q=s["q"], max_path=s["nodes"])
        return v.keep, v.path, v.token, v.delta
    caches = [paged.PagedCache(codes, scales) for codes, scales in s["data"]]
    if s["op"] == "compact":
        draft.paged_compact(caches, s["table"], s["lens"], s["cu"], s["path"], s["keep"])
        return s["data"]
    f = draft.page_fork(s["source"], s["lens"], s["table"], s["shares"], s["free"], s["n_free"], s["page"])
    draft.page_copy(caches, f.src, f.dst, f.rows)
    draft.page_free(s["ends"], s["lens"], s["table"], s["shares"], s["free"], s["n_free"], s["page"])
    return f.src, f.dst, f.rows, s["lens"], s["table"], s["shares"], s["free"], s["n_free"], s["data"]


def _tree(s):
    nodes, heads, page = s["nodes"], s["heads"], s["page"]
    lens, cu, parent = s["lens"].long(), s["cu"].long(), s["parent"].long()
    r = torch.arange(parent.shape[0], device=DEV)
    b = torch.searchsorted(cu[1:], r, right=True)
    first, count = cu[b], cu[1:] - cu[:-1]
    # each node's way up to the root
    words = -(-nodes // 32)
    bits = torch.zeros((parent.shape[0], 32 * words), dtype=torch.bool, device=DEV)
    at, pos = r - first, (lens - count)[b]
    for _ in range(nodes):
        live = at >= 0
        bits[r, at.clamp(min=0)] |= live
        at = torch.where(live, parent[first + at.clamp(min=0)], -1)
        pos = pos + (at >= 0)
    seen = (bits.view(-1, words, 32).long() << torch.arange(32, device=DEV)).sum(-1).int()

    # requests padded to the largest tree: [request, node x head, channel]
    t = s["table"].clamp(min=0)
    k = _values(s["codes"][t], s["scales"][t] if s["scales"] is not None else None, s["fmt"]).flatten(1, 2)
    i, j = torch.arange(nodes, device=DEV), torch.arange(k.shape[1], device=DEV)
    row = (cu[:-1, None] + i).clamp(max=parent.shape[0] - 1)
    q = s["q"].float()[row].flatten(1, 2)
    node = j - (lens - count)[:, None]                       # a key's node, below 0 for what was there before
    inside = node.clamp(0, nodes - 1)
    drafted = bits[row].gather(2, inside[:, None].expand(-1, nodes, -1)) & (node < count[:, None])[:, None]
    see = torch.where((node < 0)[:, None], True, drafted)
    if s["window"]:
        key_pos = torch.where(node < 0, j, pos[row].gather(1, inside))
        see &= key_pos[:, None] > (pos[row] - s["window"])[..., None]
    logit = (q @ k.mT * s["scale"]).unflatten(1, (nodes, heads)).masked_fill_(~see[:, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = logit.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1)
    o = (p.flatten(1, 2) @ k[..., :s["dv"]]).unflatten(1, (nodes, heads)) / torch.where(total > 0, total, 1.0)[..., None]
    lse = torch.where(total > 0, top[..., 0] + total.log(), -math.inf)
    return pos.int(), seen, o[b, r - first].bfloat16(), lse[b, r - first]


def _whole(w):
    """Weights from 0 to 1 as whole numbers: multiples of 2^-40, the nearest, ties to even."""
    return (w.clamp(max=1.0) * 2.0 ** 40).round().long()


def _verify(s):
    """One sweep over the nodes: a node whose parent is the kept node is tried.  What is left of the target's row p after a rejection
    is max(p - c q, 0) of mass `left`: c grows by the mass before.  Without q the tried token's probability goes.  Each float32
    operation rounds once; sums are whole numbers."""
    p, drafted, nodes = s["p"], s["q"], s["nodes"]
    cu, parent, token = s["cu"].long(), s["parent"].long(), s["token"].long()
    first, count = cu[:-1], cu[1:] - cu[:-1]
    B, last = first.shape[0], parent.shape[0] - 1
    at, keep = torch.zeros_like(first), torch.ones_like(first)
    c, left = torch.zeros(B, device=DEV), torch.ones(B, device=DEV)
    gone = torch.zeros((B, p.shape[1]), dtype=torch.bool, device=DEV) if drafted is None else None
    path = torch.full((B, nodes), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = 0
    b = torch.arange(B, device=DEV)
    for i in range(1, nodes):
        row = (first + i).clamp(max=last)
        tried = (i < count) & (parent[row] == at)
        x, u, here = token[row], s["u"][row], first + at
        px = p[here, x].float()
        if drafted is not None:
            qx = drafted[here, x].float()
            yes = tried & (u * qx * left < (px - c * qx).clamp(min=0.0))
            no = tried & ~yes
            c = torch.where(no, c + left, c)
            rest = (p[here].float() - c[:, None] * drafted[here].float()).clamp(min=0.0)
            left = torch.where(no, _whole(rest).sum(1).float() * 2.0 ** -40, left)
        else:
            px = torch.where(gone[b, x], 0.0, px)
            yes = tried & (u * left < px)
            no = tried & ~yes
            left = torch.where(no, (left - px).clamp(min=0.0), left)
            gone[b, x] |= no
            gone &= ~yes[:, None]
        path[b, keep.clamp(max=nodes - 1)] = torch.where(yes, i, path[b, keep.clamp(max=nodes - 1)])
        keep = keep + yes
        at = torch.where(yes, i, at)
        c, left = torch.where(yes, 0.0, c), torch.where(yes, 1.0, left)
    rows = p[first + at].float()
    w = rows.masked_fill(gone, 0.0) if drafted is None else (rows - c[:, None] * drafted[first + at].float()).clamp(min=0.0)
    w = _whole(w)
    w = torch.where((w.sum(1) > 0)[:, None], w, _whole(rows))
    below = w.cumsum(1)
    m = (s["r"] * 2.0 ** 24).floor().long().clamp(0, (1 << 24) - 1)
    total = below[:, -1]
    aim = (total >> 24) * m + ((total & ((1 << 24) - 1)) * m >> 24)
    token = (below <= aim[:, None]).sum(1)
    return keep.int(), path.int(), token.int(), (keep - count).int()


def _compact(s):
    page, cu = s["page"], s["cu"].long()
    base = s["lens"].long() - (cu[1:] - cu[:-1])
    i = torch.arange(s["path"].shape[1], device=DEV)
    real = i < s["keep"][:, None]
    b = torch.arange(base.shape[0], device=DEV)[:, None].expand_as(real)[real]
    src, dst = (base[:, None] + s["path"])[real], (base[:, None] + i)[real]
    src, dst = (s["table"][b, at // page].long() * page + at % page for at in (src, dst))
    for codes, scales in s["data"]:
        for t in (codes, scales):
            if t is not None:
                t.flatten(0, 1)[dst] = t.flatten(0, 1)[src]
    return s["data"]


def _fork(s):
    page, table, shares, free, lens = s["page"], s["table"], s["shares"], s["free"], s["lens"]
    source = s["source"].long()
    child = source >= 0
    up = source.clamp(min=0)
    n = torch.where(child, lens[up], 0).long()
    # full pages are shared
    j = torch.arange(table.shape[1], device=DEV)
    common = child[:, None] & (j < (n // page)[:, None])
    table.copy_(torch.where(common, table[up], table))
    shares.index_add_(0, torch.where(common, table, 0).flatten().long(), common.flatten().int())
    # the last one is copied into a page from the top of the free list, requests in order
    part = child & (n % page > 0)
    dst = free[(s["n_free"].long() - part.cumsum(0)).clamp(min=0)]
    last = (n // page).clamp(max=table.shape[1] - 1)[:, None]
    src = torch.where(part, table[up].gather(1, last)[:, 0], -1)
    dst = torch.where(part, dst, -1)
    rows = torch.where(part, n % page, 0).int()
    table.scatter_(1, last, torch.where(part[:, None], dst[:, None], table.gather(1, last)))
    s["n_free"] -= part.sum().int()
    lens.copy_(torch.where(child, n.int(), lens))
    some = torch.arange(page, device=DEV) < rows[:, None]
    at = torch.arange(page, device=DEV).expand_as(some)[some]
    a, z = (v[:, None].expand_as(some)[some].long() for v in (src, dst))
    for codes, scales in s["data"]:
        for t in (codes, scales):
            if t is not None:
                t[z, at] = t[a, at]
    # the answers end: pages that nobody holds any more go on the free list, the lowest first
    ends = s["ends"] > 0
    held = ends[:, None] & (j < (-(-lens.long() // page))[:, None]) & (table >= 0)
    shares.index_add_(0, torch.where(held, table, 0).flatten().long(), -held.flatten().int())
    nobody = shares < 0
    shares.clamp_(min=0)
    place = torch.where(nobody, s["n_free"].long() + nobody.cumsum(0) - 1, free.shape[0])
    free.copy_(torch.cat([free, free.new_zeros(1)]).scatter(0, place, torch.arange(shares.shape[0], device=DEV).int())[:-1])
    s["n_free"] += nobody.sum().int()
    lens.masked_fill_(ends, 0)
    return src, dst, rows, lens, table, shares, free, s["n_free"], s["data"]


# ------------------------------------------------------------------------------------------ 64 bits
def _power64(e):
    """2^e in 64 bits for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


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


def exact(c, seed):
    if c["op"] != "tree":
        return None                                     # whole numbers, and bytes moved
    s = prepare(c, seed)
    sizes, parents = _trees(c)
    out = torch.zeros((sum(sizes), c["heads"], c["dv"]), dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b, (n, size, parent) in enumerate(zip(_lengths(c, sizes), sizes, parents)):
        pages = s["table"][b, :-(-n // c["page"])].long()
        k = _decode64(s["codes"][pages].flatten(0, 1)[:n], s["scales"][pages].flatten(0, 1)[:n] if s["scales"] is not None else None, c["fmt"])
        see = torch.zeros((size, n), dtype=torch.bool)
        for i in range(size):
            way = [i]
            while parent[way[-1]] >= 0:
                way.append(parent[way[-1]])
            low = n - size + len(way) - c["window"] if c["window"] else 0
            see[i, max(0, low):n - size] = True
            for up, node in enumerate(way):             # `up` places before the query
                see[i, n - size + node] = not c["window"] or up < c["window"]
        see = see.to(DEV)
        for at in range(0, size, 32):                   # 32 nodes at a time
            m = min(32, size - at)
            q = s["q"][first + at:first + at + m].double()
            z = (q.flatten(0, 1) @ k.T * s["scale"]).view(m, c["heads"], n).masked_fill(~see[at:at + m, None], -math.inf)
            norm = torch.logsumexp(z, -1)
            w = torch.exp(z - norm[..., None])
            out[first + at:first + at + m] = (w.flatten(0, 1) @ k[:, :c["dv"]]).view(m, c["heads"], -1)
            lse[first + at:first + at + m] = norm
        first += size
    return None, None, out, lse
