"""The packed calls at their edges: waits that run out, tables and lengths at their limits,
streams given by argument, NaN, and the accuracy that the header states."""

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, f64, need_gpu
from test_gpu_prompt import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


@pytest.fixture
def wait_limit():
    """Sets the limit of the device's waits; the default comes back after the test."""
    yield lambda ns: binding.lib().kv_set_wait_limit_ns(ns)
    binding.lib().kv_set_wait_limit_ns(2_000_000_000)


# ------------------------------------------------------------------ waits that run out

def long_items(D, tokens):
    """One row per sequence over a table that names the same few pages again and again: the KV
    heads are items of tokens / 128 key tiles each, one after the other with num_shares = 1."""
    c = Case((1,), (200,), "bf16", D, 4, PS=64)
    table = c.table[0, torch.arange(tokens // 64, device="cuda") % 3].view(1, -1).contiguous()
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    c.kv = skv.PagedKV(c.k_pool, c.v_pool, table, lens)
    return c


@pytest.mark.parametrize("D", [128, 64])
def test_waits_that_run_out_are_flagged_and_end_the_call(wait_limit, D):
    """Without any patience the second item's rows, which wait for the first item's end, are given
    up, and every warp with them: the call says so and ends, and the next one is as ever."""
    c = long_items(D, 1 << 22)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=1)
    assert_no_device_error()
    for _ in range(3):
        wait_limit(0)
        skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=1)
        wait_limit(2_000_000_000)
        assert skv.kv_check_device_errors() == (-6, 16)
        out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=1)
        assert_no_device_error()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("limit", [50_000, 2 ** 64 - 1])
def test_long_items_do_not_run_out_of_a_copy_s_limit(wait_limit, limit, D):
    """The limit is for copies: 2^22 keys keep a block busy for 40 ms, each copy for microseconds.
    The largest limit there is does not wrap round."""
    c = long_items(D, 1 << 22)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=1)
    assert_no_device_error()
    wait_limit(limit)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=1)
    wait_limit(2_000_000_000)
    assert_no_device_error()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("new,past,D,G,PS,shares", [
    ((700, 1, 129, 64), (0, 2000, 90, 33), 128, 4, 16, 0),
    ((700, 1, 129, 64), (0, 2000, 90, 33), 64, 8, 32, 1),
    ((5, 2, 1), (3000, 1234, 4001), 128, 8, 64, 7),
])
def test_under_any_wait_limit_the_bits_are_right_or_flagged(wait_limit, new, past, D, G, PS,
                                                            shares):
    """A call under a short limit either says that a wait ran out or gives the usual bits; it
    writes to no row of nobody."""
    c = Case(new, past, "bf16", D, G, PS=PS, tail=3)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares)
    assert_no_device_error()
    for limit in (0, 1, 1000, 8000):
        for _ in range(4):
            out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
            lse = torch.full(c.q.shape[:2], -9.0, device="cuda")
            wait_limit(limit)
            skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares, out=out,
                                lse=lse)
            wait_limit(2_000_000_000)
            st, flags = skv.kv_check_device_errors()
            assert (st, flags) in ((0, 0), (-6, 16))
            if st == 0:
                assert torch.equal(out[:c.T], ref[:c.T]) and torch.equal(lse[:c.T], ref_lse[:c.T])
            assert (out[c.T:] == -9.0).all() and (lse[c.T:] == -9.0).all()
