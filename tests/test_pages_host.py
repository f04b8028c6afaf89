"""Outputs of the page calls that overlap their inputs are refused: no launch happens here."""

import pytest

from sparse_kv_cache_build_gb300 import binding
from sparse_kv_cache_build_gb300 import build as builder

from test_drafts_host import compact
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
