"""Refusals of the calls for drafts, windows and pages: no launch happens here."""

import ctypes
import math

import pytest

from sparse_kv_cache_build_gb300 import binding
from sparse_kv_cache_build_gb300 import build as builder

from test_prompt_host import desc

NULL = None


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.lib()


def masked(lib, name, d=None, **kw):
    a = dict(q=512, q_stride=1024, Hq=8, parents=64, cu=64, total=3, scale=0.1, window=5, sinks=0,
             shares=1, out=1024, lse=NULL, ws=NULL, bytes=0)
    a.update(kw)
    d = ctypes.byref(d or desc())
    if name == "tree":
        return lib.kv_tree_attn(d, a["q"], a["q_stride"], a["Hq"], a["parents"], a["cu"],
                                a["total"], a["scale"], a["shares"], a["out"], a["lse"], a["ws"],
                                a["bytes"], NULL)
    return lib.kv_window_attn(d, a["q"], a["q_stride"], a["Hq"], a["cu"], a["total"], a["scale"],
                              a["window"], a["sinks"], a["shares"], a["out"], a["lse"], a["ws"],
                              a["bytes"], NULL)


@pytest.mark.parametrize("name", ["tree", "window"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=NULL), -1), (dict(out=NULL), -1), (dict(total=-1), -1), (dict(cu=NULL), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(shares=-1), -1), (dict(shares=1025), -1), (dict(Hq=6), -2),
    (dict(Hq=7), -1), (dict(q_stride=1016), -1), (dict(q_stride=1028), -7), (dict(q=520), -7),
    (dict(out=1032), -7), (dict(total=0), 0),
])
def test_masked_attention_refusals(lib, name, kw, status):
    assert masked(lib, name, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), -1), (dict(window=-3), -1), (dict(sinks=-1), -1),
    (dict(window=1, total=0), 0), (dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1, total=0), 0),
])
def test_window_refusals(lib, kw, status):
    assert masked(lib, "window", **kw) == status


def test_a_tree_needs_parents(lib):
    assert masked(lib, "tree", parents=NULL) == -1
    assert lib.kv_tree_attn(None, 512, 1024, 8, 64, 64, 3, 0.1, 1, 1024, NULL, NULL, 0, NULL) == -1
    assert lib.kv_window_attn(None, 512, 1024, 8, 64, 3, 0.1, 1, 0, 1, 1024, NULL, NULL, 0,
                              NULL) == -1


@pytest.mark.parametrize("name", ["tree", "window"])
def test_masked_attention_caches(lib, name):
    assert masked(lib, name, desc(head_dim=96)) == -2
    assert masked(lib, name, desc(page_size=8)) == -2
    assert masked(lib, name, desc(k_pool=NULL)) == -1
    last = (2 ** 31 - 1 - 256) // 16
    for stride, status in ((last, 0), (last + 1, -2)):
        assert masked(lib, name, desc(page_table_stride=stride), total=0) == status
    # TMA counts a pool's rows in 32 bits
    assert masked(lib, name, desc(num_phys_pages=2 ** 26)) == -2


def compact(lib, d=None, **kw):
    a = dict(cu=64, keep=128, stride=4, cnt=256, stats=512, lens=1024)
    a.update(kw)
    return lib.kv_compact(ctypes.byref(d or desc()), a["cu"], a["keep"], a["stride"], a["cnt"],
                          a["stats"], a["lens"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(keep=NULL), -1), (dict(stride=0), -1), (dict(stride=-4), -1), (dict(cnt=NULL), -1),
    (dict(lens=NULL), -1), (dict(lens=8192), -1),          # the cache's own lengths
    (dict(stats=520), -7),
])
def test_compact_refusals(lib, kw, status):
    assert compact(lib, **kw) == status


def test_compact_caches(lib):
    assert compact(lib, desc(head_dim=96)) == -2
    assert compact(lib, desc(page_table=NULL)) == -1
    assert compact(lib, desc(page_table_stride=(2 ** 31 - 4096) // 16)) == -2


def copy(lib, d=None, **kw):
    a = dict(pairs=64, n=2, stats=512)
    a.update(kw)
    return lib.kv_copy_pages(ctypes.byref(d or desc()), a["pairs"], a["n"], a["stats"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(pairs=NULL), -1), (dict(n=-1), -1), (dict(pairs=68), -7), (dict(stats=520), -7),
    (dict(n=2 ** 31 - 1), -2), (dict(n=0), 0), (dict(n=0, pairs=NULL, stats=NULL), 0),
])
def test_copy_pages_refusals(lib, kw, status):
    assert copy(lib, **kw) == status


def update(lib, d=None, **kw):
    a = dict(refs=64, parents=NULL, rows=1, keep=NULL, new=256, window=0, sinks=0, table=65536,
             copies=512, left=1024)
    a.update(kw)
    return lib.kv_update_pages(ctypes.byref(d or desc()), a["refs"], a["parents"], a["rows"],
                               a["keep"], a["new"], a["window"], a["sinks"], a["table"],
                               a["copies"], a["left"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(refs=NULL), -1), (dict(new=NULL), -1), (dict(table=NULL), -1), (dict(copies=NULL), -1),
    (dict(left=NULL), -1), (dict(rows=0), -1), (dict(rows=2), -1), (dict(window=-1), -1),
    (dict(sinks=-1), -1), (dict(rows=16385, parents=64), -2), (dict(refs=68), -7),
    # in place only where a row continues itself
    (dict(table=4096, parents=64), -1), (dict(table=4100), -1), (dict(table=4096 - 4), -1),
    (dict(table=4096 - 16, parents=64, rows=2), -1),
])
def test_update_pages_refusals(lib, kw, status):
    assert update(lib, **kw) == status


def test_update_pages_caches(lib):
    assert update(lib, desc(batch=16385), rows=5, parents=64) == -2
    assert update(lib, desc(page_size=8)) == -2
    assert update(lib, desc(page_table_stride=(2 ** 31 - 256) // 16)) == -2
