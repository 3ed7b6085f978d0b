"""The paged-cache calls on the host: exported symbols, a plain C header, formats told from
widths, and every refusal (none of these calls reaches the GPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from fp4_kv_cache_gb300 import build as libbuild
from fp4_kv_cache_gb300 import csa2, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096                    # never dereferenced: the calls below fail validation first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return paged._lib()


def test_exports_the_header(lib):
    src = open(os.path.join(ROOT, "include", "csa2_paged.h")).read()
    declared = set(re.findall(r"CSA2_API[^;(]*?\b(csa2p_\w+)\s*\(", src))
    out = os.popen(f"nm -D --defined-only {libbuild.LIB}").read()
    assert declared == set(re.findall(r" T (csa2p_\w+)", out)) and len(declared) == 6


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "use_paged.c"
    src.write_text('#include "csa2_paged.h"\n#include <stdio.h>\n'
                   'int main(void) {\n'
                   '    printf("%zu %zu %zu %zu\\n", sizeof(csa2p_cache), sizeof(csa2p_plan_args),\n'
                   '           sizeof(csa2p_rope_axes), sizeof(csa2p_attn_args));\n'
                   '    return 0;\n}\n')
    exe = tmp_path / "use_paged"
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    sizes = subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()
    assert [int(s) for s in sizes] == [ctypes.sizeof(t) for t in (paged.CacheArgs, paged.PlanArgs, paged.RopeAxes,
                                                                  paged.AttnArgs)]


def cache(**k):
    v = dict(fmt=paged.MXFP4, d=576, page=64, n_pages=10, codes=FAKE, scales=FAKE, code_stride=0, scale_stride=0)
    v.update(k)
    return paged.CacheArgs(*(v[n] for n, _ in paged.CacheArgs._fields_))


BAD_CACHES = [dict(fmt=4), dict(fmt=-1), dict(d=0), dict(d=48), dict(d=1056), dict(page=0), dict(page=48),
              dict(page=1 << 17), dict(n_pages=-1), dict(n_pages=1 << 25), dict(codes=None), dict(codes=FAKE + 8),
              dict(scales=None), dict(code_stride=64 * 288 - 16), dict(code_stride=64 * 288 + 8),
              dict(scale_stride=64 * 18 - 2)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_caches_refused(lib, bad):
    c = ctypes.byref(cache(**bad))
    assert lib.csa2p_write(c, FAKE, 576, 4, FAKE, None, None, None) == INVALID
    assert lib.csa2p_read(c, FAKE, 4, FAKE, 576, None, None) == INVALID
    a = attn(cache=cache(**bad))
    assert lib.csa2p_attn_workspace_size(ctypes.byref(a)) == 0
    assert lib.csa2p_attn(ctypes.byref(a), FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID


def test_write_and_read_refused(lib):
    c = ctypes.byref(cache())
    w, r = lib.csa2p_write, lib.csa2p_read
    assert w(None, FAKE, 576, 4, FAKE, None, None, None) == INVALID
    assert w(c, FAKE, 576, -1, FAKE, None, None, None) == INVALID
    assert w(c, None, 576, 4, FAKE, None, None, None) == INVALID
    assert w(c, FAKE, 576, 4, None, None, None, None) == INVALID
    assert w(c, FAKE + 8, 576, 4, FAKE, None, None, None) == INVALID       # rows not 16-byte aligned
    assert w(c, FAKE, 580, 4, FAKE, None, None, None) == INVALID
    assert w(c, FAKE, 568, 4, FAKE, None, None, None) == INVALID           # rows overlap
    assert w(c, None, 0, 0, None, None, None, None) == 0                   # nothing to do
    assert r(None, FAKE, 4, FAKE, 576, None, None) == INVALID
    assert r(c, None, 4, FAKE, 576, None, None) == INVALID
    assert r(c, FAKE, 4, None, 576, None, None) == INVALID
    assert r(c, FAKE, 4, FAKE, 572, None, None) == INVALID
    assert r(c, FAKE, 4, FAKE, 568, None, None) == INVALID
    assert r(c, None, 0, None, 0, None, None) == 0


def rope(dim=64, axes=1, sec=(32, 0, 0), pos=FAKE, cs=FAKE, n_pos=10):
    return paged.RopeAxes(dim, axes, (ctypes.c_int32 * 3)(*sec), pos, cs, n_pos)


BAD_ROPES = [rope(dim=63), rope(dim=-2), rope(dim=578, sec=(289, 0, 0)), rope(axes=0), rope(axes=4), rope(sec=(31, 0, 0)),
             rope(axes=2, sec=(40, -8, 0)), rope(axes=2, sec=(16, 8, 8)), rope(pos=None), rope(cs=None), rope(n_pos=0)]


@pytest.mark.parametrize("i", range(len(BAD_ROPES)))
def test_rotations_refused(lib, i):
    r = ctypes.byref(BAD_ROPES[i])
    assert lib.csa2p_rope(FAKE, 576, 576, FAKE, 576, 576, 4, 1, 576, r, None, None) == INVALID
    assert lib.csa2p_write(ctypes.byref(cache()), FAKE, 576, 4, FAKE, r, None, None) == INVALID


def test_rope_refused(lib):
    f, r = lib.csa2p_rope, ctypes.byref(rope())
    other = FAKE + (1 << 20)
    assert f(FAKE, 1152, 576, other, 1152, 576, -1, 2, 576, r, None, None) == INVALID
    assert f(FAKE, 1152, 576, other, 1152, 576, 4, 2, 572, r, None, None) == INVALID      # d % 8
    assert f(None, 1152, 576, other, 1152, 576, 4, 2, 576, r, None, None) == INVALID
    assert f(FAKE, 1152, 576, None, 1152, 576, 4, 2, 576, r, None, None) == INVALID
    assert f(FAKE + 8, 1152, 576, other, 1152, 576, 4, 2, 576, r, None, None) == INVALID
    assert f(FAKE, 1156, 576, other, 1152, 576, 4, 2, 576, r, None, None) == INVALID      # strides % 8
    assert f(FAKE, 1152, 576, other, 1152, 568, 4, 2, 576, r, None, None) == INVALID      # heads overlap in out
    assert f(FAKE, 1152, 576, other, 568, 576, 4, 2, 576, r, None, None) == INVALID       # rows overlap in out
    assert f(FAKE, 1152, 576, FAKE, 1160, 576, 4, 2, 576, r, None, None) == INVALID       # in place, other strides
    assert f(None, 0, 0, None, 0, 0, 0, 2, 576, None, None, None) == 0


def plan(**k):
    v = dict(batch=4, page=64, width=10, free_cap=20, n_rows=8, lens=FAKE, delta=FAKE, lens_out=FAKE, block_table=FAKE,
             free_pages=FAKE, n_free=FAKE, n_free_out=FAKE, cu=FAKE, slot=FAKE, row_req=FAKE, row_pos=FAKE)
    v.update(k)
    return ctypes.byref(paged.PlanArgs(*(v[n] for n, _ in paged.PlanArgs._fields_)))


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(batch=paged.MAX_BATCH + 1), dict(page=0), dict(page=3),
                                 dict(page=1 << 17), dict(width=0), dict(free_cap=-1), dict(n_rows=-1)]
                         + [{n: None} for n in ("lens", "delta", "lens_out", "block_table", "free_pages", "n_free",
                                                "n_free_out", "cu", "slot")], ids=str)
def test_plans_refused(lib, bad):
    assert lib.csa2p_page_plan(plan(**bad), None, None) == INVALID
    assert lib.csa2p_page_plan(None, None, None) == INVALID


def attn(**k):
    v = dict(cache=cache(), batch=2, n_tokens=4, n_heads=64, d_v=512, width=5, window=0, ratio_m=1, sm_scale=0.04,
             q=FAKE, block_table=FAKE, lens=FAKE, cu=FAKE, pos0=FAKE, kv_start=FAKE)
    v.update(k)
    return paged.AttnArgs(*(v[n] for n, _ in paged.AttnArgs._fields_))


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), INVALID), (dict(batch=paged.MAX_BATCH + 1), INVALID), (dict(n_tokens=-1), INVALID),
    (dict(n_heads=0), INVALID), (dict(n_heads=129), INVALID), (dict(d_v=0), INVALID), (dict(d_v=508), INVALID),
    (dict(d_v=584), INVALID), (dict(d_v=520), UNSUPPORTED), (dict(cache=cache(d=640)), UNSUPPORTED),
    (dict(cache=cache(n_pages=1 << 22)), UNSUPPORTED), (dict(cache=cache(code_stride=1 << 33)), UNSUPPORTED),
    (dict(cache=cache(scale_stride=1 << 29)), UNSUPPORTED), (dict(width=-1), INVALID), (dict(window=-1), INVALID), (dict(ratio_m=0), INVALID), (dict(sm_scale=0.0), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(sm_scale=float("inf")), INVALID), (dict(q=None), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(block_table=None), INVALID), (dict(lens=None), INVALID), (dict(cu=None), INVALID),
    (dict(pos0=None, ratio_m=2), INVALID), (dict(n_tokens=1 << 25), INVALID)], ids=str)
def test_attn_refused(lib, bad, status):
    a = ctypes.byref(attn(**bad))
    assert lib.csa2p_attn_workspace_size(a) == 0
    assert lib.csa2p_attn(a, FAKE, FAKE, FAKE, 1 << 40, None, None) == status


def test_attn_outputs_refused_and_empty(lib):
    a = ctypes.byref(attn())
    assert lib.csa2p_attn(a, None, FAKE, FAKE, 1 << 40, None, None) == INVALID
    assert lib.csa2p_attn(a, FAKE + 8, FAKE, FAKE, 1 << 40, None, None) == INVALID
    assert lib.csa2p_attn(None, FAKE, FAKE, FAKE, 1 << 40, None, None) == INVALID
    need = lib.csa2p_attn_workspace_size(a)
    if need:
        assert lib.csa2p_attn(a, FAKE, FAKE, FAKE, need - 1, None, None) == WORKSPACE
        assert lib.csa2p_attn(a, FAKE, FAKE, None, need, None, None) == INVALID
        assert lib.csa2p_attn(a, FAKE, FAKE, FAKE + 8, need, None, None) == INVALID
    for empty in (attn(batch=0), attn(n_tokens=0)):
        assert lib.csa2p_attn(ctypes.byref(empty), None, None, None, 0, None, None) == 0


def test_formats_from_widths():
    for fmt in (paged.MXFP4, paged.NVFP4_E4M3_16, paged.MXFP8, paged.BF16):
        c = paged.PagedCache.new(3, 16, 576, fmt, device="cpu")
        assert (c.fmt, c.d, c.page, c.n_pages) == (fmt, 576, 16, 3)
    wide = torch.zeros((6, 2, 16, 288), dtype=torch.uint8)                 # two layers' pages side by side
    c = paged.PagedCache(wide[:, 1], torch.zeros((6, 16, 18), dtype=torch.uint8))
    assert c.fields[-2:] == (2 * 16 * 288, 16 * 18)


def test_binding_refuses(lib):
    u8 = torch.uint8
    with pytest.raises(ValueError):
        paged.PagedCache(torch.zeros((3, 16, 288), dtype=u8), torch.zeros((3, 16, 20), dtype=u8))
    with pytest.raises(ValueError):
        paged.PagedCache(torch.zeros((3, 16, 288), dtype=u8))              # bytes without scales
    with pytest.raises(ValueError):
        paged.PagedCache(torch.zeros((3, 16, 576), dtype=u8)[:, :, ::2], torch.zeros((3, 16, 18), dtype=u8))
    c = paged.PagedCache.new(3, 16, 64, device="cpu")
    i32 = torch.int32
    with pytest.raises(ValueError):
        paged.paged_write(c, torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        paged.paged_read(c, torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        paged.paged_attn(torch.zeros((2, 4, 64), dtype=torch.bfloat16), c, torch.zeros((1, 3), dtype=i32),
                         torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        paged.page_plan(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros((2, 3), dtype=i32),
                        torch.zeros(4, dtype=i32), torch.zeros(1, dtype=i32), 16, 4)
    with pytest.raises(ValueError):
        paged.rope_axes(torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=i32), torch.zeros((9, 32)))


def test_packed_structures():
    # the packed argument structures lie as the ctypes (and so the C) ones do
    for packer, cls in ((paged._CACHE, paged.CacheArgs), (paged._PLAN, paged.PlanArgs), (paged._ROPE, paged.RopeAxes),
                        (paged._ATTN, paged.AttnArgs)):
        assert packer.size == ctypes.sizeof(cls)
    c = paged.PagedCache.new(3, 16, 576, paged.NVFP4_E4M3_16, device="cpu")
    a = paged.CacheArgs.from_buffer_copy(c.packed)
    assert [getattr(a, n) or 0 for n, _ in a._fields_] == list(c.fields)
    v = list(range(1, 17))
    a = paged.PlanArgs.from_buffer_copy(paged._PLAN.pack(*v))
    assert [getattr(a, n) for n, _ in a._fields_] == v
    a = paged.RopeAxes.from_buffer_copy(paged._ROPE.pack(*v[:8]))
    assert (a.rope_dim, a.n_axes, list(a.section), a.pos, a.cos_sin, a.n_pos) == (1, 2, [3, 4, 5], 6, 7, 8)
    a = paged.AttnArgs.from_buffer_copy(paged._ATTN.pack(*c.fields, *v[:7], 0.5, *v[8:14]))
    assert [getattr(a, n) for n, _ in a._fields_[1:]] == v[:7] + [0.5] + v[8:14]


def test_status_text():
    assert "invalid" in csa2.status_string(INVALID)
