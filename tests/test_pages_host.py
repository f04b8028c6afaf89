"""Outputs of the page calls that overlap their inputs are refused: no launch happens here."""

import pytest

from sparse_kv_cache_build_gb300 import binding
from sparse_kv_cache_build_gb300 import build as builder

from test_drafts_host import compact, update
from test_prompt_host import desc


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.lib()


B = 3       # sequences; addresses: cu 64 (4 words), keep 128 (12), keep_cnt 256 (3)


@pytest.mark.parametrize("lens", [
    256, 252, 264,                  # the counts, and a word before and behind their first
    128, 172, 120,                  # the kept indices
    64, 76, 56,                     # the offsets
    8192, 8200, 8184,               # the sequences' lengths
    4096, 4140,                     # the page table (12 words)
])
def test_compact_refuses_lengths_over_its_inputs(lib, lens):
    assert compact(lib, desc(batch=B), lens=lens) == -1


# four pages, old rows of four entries; three new rows
LISTS = dict(parents=16384, keep=20480, new=24576, refs=64, table=65536, copies=512, left=1024)


@pytest.mark.parametrize("kw", [
    dict(copies=16384), dict(copies=16400 - 24), dict(left=16392), dict(table=16384 - 44),
    dict(copies=20480), dict(left=20488), dict(left=24576), dict(copies=24580), dict(refs=24576),
    dict(left=8192), dict(copies=8192 - 20), dict(table=8192), dict(refs=8192),
    dict(left=4096), dict(copies=4096 + 12), dict(refs=4096),
    dict(left=64), dict(left=76), dict(copies=64), dict(table=80 - 4), dict(refs=65536),
    dict(left=512), dict(left=532), dict(copies=65536 + 44), dict(left=65536 + 44),
    dict(left=65536, table=65536, copies=65536),
])
def test_update_pages_refuses_outputs_over_inputs_and_each_other(lib, kw):
    assert update(lib, desc(), rows=3, **{**LISTS, **kw}) == -1


def test_update_pages_in_place_still_overlaps_nothing_else(lib):
    for kw in (dict(left=4096), dict(copies=4104), dict(refs=4096), dict(new=4100)):
        assert update(lib, **{**dict(table=4096), **kw}) == -1
