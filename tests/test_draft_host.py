"""The calls for drafted tokens and shared pages on the host: exported symbols, a plain C header, and
every refusal (none of these calls reaches the GPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from fp4_kv_cache_gb300 import build as libbuild
from fp4_kv_cache_gb300 import draft, paged
from test_paged_host import BAD_CACHES, FAKE, INVALID, ROOT, UNSUPPORTED, WORKSPACE, cache

OFF = FAKE + 2                  # no address of 32-bit values
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return draft._lib()


def test_exports_the_header(lib):
    src = open(os.path.join(ROOT, "include", "csa2_draft.h")).read()
    declared = set(re.findall(r"CSA2_API[^;(]*?\b(csa2d_\w+)\s*\(", src))
    out = os.popen(f"nm -D --defined-only {libbuild.LIB}").read()
    assert declared == set(re.findall(r" T (csa2d_\w+)", out)) and len(declared) == 8


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "use_draft.c"
    src.write_text('#include "csa2_draft.h"\n#include <stdio.h>\n'
                   'int main(void) {\n'
                   '    printf("%zu %zu %zu %zu %zu\\n", sizeof(csa2d_tree_args), sizeof(csa2d_tree_attn_args),\n'
                   '           sizeof(csa2d_verify_args), sizeof(csa2d_compact_args), sizeof(csa2d_share_args));\n'
                   '    return 0;\n}\n')
    exe = tmp_path / "use_draft"
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    sizes = [int(s) for s in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert sizes == [ctypes.sizeof(t) for t in (draft.TreeArgs, draft.TreeAttnArgs, draft.VerifyArgs, draft.CompactArgs, draft.ShareArgs)]
    assert sizes == [t.size for t in (draft._TREE, draft._ATTN, draft._VERIFY, draft._COMPACT, draft._SHARE)]


def make(kind, defaults, k):
    v = dict(defaults)
    v.update(k)
    return kind(*(v.get(n, FAKE) for n, _ in kind._fields_))


def tree(**k):
    return ctypes.byref(make(draft.TreeArgs, dict(batch=2, n_tokens=8, words=1), k))


def attn(**k):
    return ctypes.byref(make(draft.TreeAttnArgs, dict(cache=cache(), batch=2, n_tokens=8, n_heads=64, d_v=512, width=4, window=0, words=1,
                                                      sm_scale=0.04), k))


def verify(**k):
    return ctypes.byref(make(draft.VerifyArgs, dict(batch=2, n_tokens=8, vocab=100, type=0, max_path=4, p_row=100, q_row=100), k))


def compact(**k):
    return ctypes.byref(make(draft.CompactArgs, dict(batch=2, width=4, max_path=4), k))


def share(**k):
    return ctypes.byref(make(draft.ShareArgs, dict(batch=2, page=64, width=4, n_pages=10, free_cap=10), k))


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(n_tokens=-1), dict(words=0), dict(words=33), dict(pos=None),
                                 dict(seen=None), dict(parent=None), dict(lens=None), dict(cu=None), dict(pos=OFF), dict(seen=OFF), dict(parent=OFF),
                                 dict(lens=OFF), dict(cu=OFF)], ids=str)
def test_tree_plan_refused(lib, bad):
    assert lib.csa2d_tree_plan(tree(**bad), None, None) == INVALID


def test_tree_plan_others(lib):
    assert lib.csa2d_tree_plan(None, None, None) == INVALID
    assert lib.csa2d_tree_plan(tree(), OFF, None) == INVALID
    assert lib.csa2d_tree_plan(tree(n_tokens=0, parent=None, pos=None, seen=None), None, None) == 0


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(n_tokens=-1), dict(n_heads=0), dict(n_heads=129), dict(d_v=0),
                                 dict(d_v=12), dict(d_v=584), dict(width=-1), dict(window=-1), dict(words=0), dict(words=33), dict(sm_scale=0.0),
                                 dict(sm_scale=float("nan")), dict(sm_scale=2.4e38), dict(n_tokens=1 << 26), dict(q=None), dict(q=FAKE + 8), dict(lens=None),
                                 dict(cu=None), dict(seen=None), dict(block_table=None), dict(window=5, pos=None), dict(block_table=OFF),
                                 dict(lens=OFF), dict(cu=OFF), dict(seen=OFF), dict(pos=OFF), dict(kv_start=OFF)], ids=str)
def test_tree_attn_refused(lib, bad):
    assert lib.csa2d_tree_attn_workspace_size(attn(**bad)) == 0
    assert lib.csa2d_tree_attn(attn(**bad), FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_caches_refused(lib, bad):
    c = cache(**bad)
    assert lib.csa2d_tree_attn(attn(cache=c), FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID
    both = (paged.CacheArgs * 2)(cache(), c)
    assert lib.csa2d_compact(compact(), both, 2, None, None) == INVALID
    assert lib.csa2d_page_copy(both, 2, FAKE, FAKE, FAKE, 3, None, None) == INVALID


def test_tree_attn_others(lib):
    f, size = lib.csa2d_tree_attn, lib.csa2d_tree_attn_workspace_size
    assert size(None) == 0 and f(None, FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID
    assert f(attn(cache=cache(d=608)), FAKE, FAKE, FAKE, 1 << 40, None, None) == UNSUPPORTED
    assert f(attn(cache=cache(d=1024), d_v=520), FAKE, FAKE, FAKE, 1 << 40, None, None) == UNSUPPORTED
    assert f(attn(), None, FAKE, FAKE, 1 << 40, None, None) == INVALID
    assert f(attn(), FAKE + 8, FAKE, FAKE, 1 << 40, None, None) == INVALID
    assert f(attn(), FAKE, OFF, FAKE, 1 << 40, None, None) == INVALID
    assert f(attn(), FAKE, FAKE, FAKE, 1 << 40, OFF, None) == INVALID
    need = size(attn())
    if need:                                                               # (no GPU: no multiprocessors, no parts)
        assert f(attn(), FAKE, FAKE, FAKE, need - 1, None, None) == WORKSPACE
        assert f(attn(), FAKE, FAKE, None, need, None, None) == INVALID
        assert f(attn(), FAKE, FAKE, FAKE + 8, need, None, None) == INVALID
    for empty in (dict(batch=0), dict(n_tokens=0)):
        assert f(attn(q=None, seen=None, lens=None, **empty), None, None, None, 0, None, None) == 0


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(n_tokens=-1), dict(vocab=0), dict(vocab=draft.MAX_VOCAB + 1), dict(type=3),
                                 dict(type=-1), dict(max_path=0), dict(p_row=99), dict(q_row=99), dict(cu=None), dict(r=None), dict(keep=None),
                                 dict(path=None), dict(next_token=None), dict(delta=None), dict(p=None), dict(token=None), dict(parent=None),
                                 dict(u=None), dict(p=OFF), dict(q=OFF), dict(p=FAKE + 1, type=1), dict(q=FAKE + 1, type=2), dict(token=OFF),
                                 dict(parent=OFF), dict(cu=OFF), dict(u=OFF), dict(r=OFF), dict(keep=OFF), dict(path=OFF), dict(next_token=OFF),
                                 dict(delta=OFF)], ids=str)
def test_verify_refused(lib, bad):
    assert lib.csa2d_tree_verify(verify(**bad), None, None) == INVALID


def test_verify_others(lib):
    assert lib.csa2d_tree_verify(None, None, None) == INVALID
    assert lib.csa2d_tree_verify(verify(), OFF, None) == INVALID
    assert lib.csa2d_tree_verify(verify(batch=0, cu=None, r=None), None, None) == 0


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(width=-1), dict(max_path=-1), dict(block_table=None), dict(lens=None),
                                 dict(cu=None), dict(path=None), dict(keep=None), dict(block_table=OFF), dict(lens=OFF), dict(cu=OFF), dict(path=OFF),
                                 dict(keep=OFF)], ids=str)
def test_compact_refused(lib, bad):
    assert lib.csa2d_compact(compact(**bad), (paged.CacheArgs * 1)(cache()), 1, None, None) == INVALID


def test_compact_others(lib):
    f, one = lib.csa2d_compact, (paged.CacheArgs * 1)(cache())
    assert f(None, one, 1, None, None) == INVALID
    assert f(compact(), one, 1, OFF, None) == INVALID
    assert f(compact(), None, 1, None, None) == INVALID
    assert f(compact(), one, -1, None, None) == INVALID
    assert f(compact(), (paged.CacheArgs * 33)(*[cache()] * 33), 33, None, None) == INVALID
    assert f(compact(), (paged.CacheArgs * 2)(cache(), cache(page=32)), 2, None, None) == INVALID
    assert f(compact(), None, 0, None, None) == 0 and f(compact(batch=0, lens=None), one, 1, None, None) == 0


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(page=0), dict(page=48), dict(page=1 << 17), dict(width=0), dict(n_pages=-1),
                                 dict(free_cap=-1), dict(n_free=None), dict(lens=None), dict(block_table=None), dict(shares=None),
                                 dict(free_pages=None), dict(lens=OFF), dict(block_table=OFF), dict(shares=OFF), dict(free_pages=OFF),
                                 dict(n_free=OFF)], ids=str)
def test_fork_and_free_refused(lib, bad):
    assert lib.csa2d_page_fork(share(**bad), None, None) == INVALID
    assert lib.csa2d_page_free(share(**bad), None, None) == INVALID


def test_fork_and_free_others(lib):
    for f, which in ((lib.csa2d_page_fork, "source"), (lib.csa2d_page_free, "ends")):
        assert f(None, None, None) == INVALID and f(share(), OFF, None) == INVALID
        assert f(share(**{which: None}), None, None) == INVALID and f(share(**{which: OFF}), None, None) == INVALID
        assert f(share(batch=0, lens=None, block_table=None, **{which: None}), None, None) == 0
    for name in ("src", "dst", "rows"):
        assert lib.csa2d_page_fork(share(**{name: None}), None, None) == INVALID
        assert lib.csa2d_page_fork(share(**{name: OFF}), None, None) == INVALID


def test_copy_refused(lib):
    f, one = lib.csa2d_page_copy, (paged.CacheArgs * 1)(cache())
    assert f(one, 1, None, FAKE, None, 3, None, None) == INVALID
    assert f(one, 1, FAKE, None, None, 3, None, None) == INVALID
    assert f(one, 1, FAKE, FAKE, None, -1, None, None) == INVALID
    for k in range(4):
        at = [FAKE] * 4
        at[k] = OFF
        assert f(one, 1, at[0], at[1], at[2], 3, at[3], None) == INVALID
    assert f(None, 1, FAKE, FAKE, None, 3, None, None) == INVALID
    assert f((paged.CacheArgs * 33)(*[cache()] * 33), 33, FAKE, FAKE, None, 3, None, None) == INVALID
    assert f(one, 1, None, None, None, 0, None, None) == 0 and f(None, 0, FAKE, FAKE, None, 3, None, None) == 0


# ------------------------------------------------------------------ the Python binding
def test_binding_refuses_cpu_tensors_and_shapes():
    i = lambda *s: torch.zeros(s, dtype=I32)                               # noqa: E731
    c = paged.PagedCache.new(2, 16, 64, device="cpu")
    for call in (lambda: draft.tree_plan(i(4), i(1), i(2), 8), lambda: draft.tree_plan(i(4), i(1), i(2), 0), lambda: draft.tree_plan(i(4), i(1), i(2), 1025),
                 lambda: draft.tree_attn(torch.zeros((4, 1, 64), dtype=torch.bfloat16), c, i(1, 1), i(1), i(2), i(4, 1)),
                 lambda: draft.tree_verify(torch.zeros((4, 9)), i(4), i(4), i(2), torch.zeros(4), torch.zeros(1)),
                 lambda: draft.tree_verify(torch.zeros((4, 9), dtype=torch.float64), i(4), i(4), i(2), torch.zeros(4), torch.zeros(1)),
                 lambda: draft.paged_compact([c], i(1, 1), i(1), i(2), i(1, 1), i(1)), lambda: draft.paged_compact([], i(1, 1), i(1), i(2), i(1, 1), i(1)),
                 lambda: draft.page_fork(i(1), i(1), i(1, 1), i(2), i(2), i(1), 16), lambda: draft.page_free(i(1), i(1), i(1, 1), i(2), i(2), i(1), 16),
                 lambda: draft.page_copy([c], i(1), i(1))):
        with pytest.raises(ValueError):
            call()
