"""The prompt operators' refusals and host-side parts: no launch happens here."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

from sparse_kv_cache_build_gb300 import binding
from sparse_kv_cache_build_gb300 import build as builder

NULL = None


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.lib()


def desc(**kw):
    base = dict(k_pool=16 * 1000, v_pool=16 * 2000, dtype=0, num_phys_pages=4,
                num_kv_heads=2, page_size=16, head_dim=128, batch=1, page_table=4096,
                page_table_stride=4, seq_lens=8192)
    base.update(kw)
    return binding.KVCacheDesc(**base)


def append(lib, d=None, **kw):
    a = dict(q=512, q_stride=1024, Hq=8, k=1024, k_stride=256, v=2048, v_stride=256, cu=64,
             total=3, positions=NULL, turns=64, rot=128, inter=0, q_out=4096, o_stride=1024,
             stats=256)
    a.update(kw)
    return lib.kv_append_rope(
        ctypes.byref(d or desc()), a["q"], a["q_stride"], a["Hq"], a["k"], a["k_stride"], a["v"],
        a["v_stride"], a["cu"], a["total"], a["positions"], a["turns"], a["rot"], a["inter"],
        a["q_out"], a["o_stride"], a["stats"], NULL)


def attn(lib, d=None, **kw):
    a = dict(q=512, q_stride=1024, Hq=8, cu=64, total=3, scale=0.1, shares=1, out=1024, lse=NULL,
             ws=NULL, bytes=0)
    a.update(kw)
    return lib.kv_prefill_attn(
        ctypes.byref(d or desc()), a["q"], a["q_stride"], a["Hq"], a["cu"], a["total"],
        a["scale"], a["shares"], a["out"], a["lse"], a["ws"], a["bytes"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(q=NULL), -1), (dict(k=NULL), -1), (dict(v=NULL), -1), (dict(q_out=NULL), -1),
    (dict(stats=NULL), -1), (dict(turns=NULL), -1), (dict(total=-1), -1),
    (dict(cu=NULL, total=3), -1),                 # one row per sequence, batch 1
    (dict(Hq=7), -1), (dict(Hq=6), -2), (dict(rot=-16), -1), (dict(rot=144), -1),
    (dict(rot=24), -2), (dict(q_stride=1016), -1), (dict(k_stride=255), -1),
    (dict(q_stride=1028), -7), (dict(v_stride=260), -7), (dict(o_stride=1025), -7),
    (dict(q=520), -7), (dict(v=2056), -7), (dict(q_out=4104), -7), (dict(stats=264), -7),
    (dict(turns=68), -7),
])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("page_size", [16, 32, 64])
def test_tables_whose_positions_pass_32_bits_are_refused(lib, page_size):
    """2^31 - 256 tokens to a table row and more: the rows of a tile may lie past the last."""
    last = (2 ** 31 - 1 - 256) // page_size
    most = (2 ** 31 - 1) // page_size
    for stride, status in ((last, 0), (last + 1, -2), (most, -2)):
        d = desc(page_size=page_size, page_table_stride=stride)
        assert append(lib, d, total=0) == status
        assert attn(lib, d, total=0) == status


def test_append_refuses_bad_caches_and_accepts_nothing_to_do(lib):
    assert append(lib, desc(head_dim=96)) == -2
    assert append(lib, desc(k_pool=NULL)) == -1
    assert append(lib, total=0) == 0
    assert append(lib, total=0, rot=0, turns=NULL) == 0
    # fp32 rows step by 16 bytes in elements of four
    assert append(lib, desc(dtype=1), total=0, q_stride=1028) == 0
    assert append(lib, desc(dtype=1), total=0, q_stride=1030) == -7


@pytest.mark.parametrize("kw,status", [
    (dict(q=NULL), -1), (dict(out=NULL), -1), (dict(total=-1), -1), (dict(cu=NULL), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(shares=-1), -1), (dict(shares=1025), -1), (dict(Hq=6), -2),
    (dict(Hq=7), -1), (dict(q_stride=1016), -1), (dict(q_stride=1028), -7), (dict(q=520), -7),
    (dict(out=1032), -7),
])
def test_attention_refusals(lib, kw, status):
    assert attn(lib, **kw) == status


def test_attention_accepts_nothing_to_do(lib):
    assert attn(lib, total=0) == 0
    assert attn(lib, desc(page_size=8), total=0) == -2


def test_workspace_size_formula(lib):
    d = desc()
    r256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for T, S in ((5, 2), (100, 7)):               # tiles of 256 rows, four heads to a token
        rows = 2 * S * min(256, T * 4)
        want = r256(rows * 128 * 4) + r256(rows * 8) + r256(24 * S)
        assert lib.kv_prefill_attn_workspace_size(ctypes.byref(d), 8, T, S) == want
        assert lib.kv_workspace_size(4, ctypes.byref(d), 8, T, S) == want
    assert lib.kv_prefill_attn_workspace_size(ctypes.byref(d), 8, 100, 1) == 0
    for bad in ((0, 5, 2), (6, 5, 2), (8, -1, 2), (8, 5, 1025), (8, 5, -1)):
        assert lib.kv_prefill_attn_workspace_size(ctypes.byref(d), *bad) == 0
    assert lib.kv_prefill_attn_workspace_size(NULL, 8, 5, 2) == 0


def test_turns_are_the_fraction_of_a_turn(lib):
    freq = [1.0, 0.0, 2 * math.pi, 1e-6, -1e-6, 7.5, 1e9]
    turns = binding.kv_rope_turns(freq)
    assert turns.dtype == torch.int64
    for f, t in zip(freq, turns.tolist()):
        want = (f / (2 * math.pi)) % 1.0
        got = (t % 2 ** 64) / 2.0 ** 64
        # one rounding of the quotient, relative to the angle's own size
        err = abs(got - want)
        assert min(err, 1 - err) <= 2 ** -53 * (1 + abs(f))
    one = (ctypes.c_double * 1)(math.nan)
    out = (ctypes.c_uint64 * 1)()
    assert lib.kv_rope_turns(one, 1, out) == -1
    assert lib.kv_rope_turns(one, 0, out) == -1
    assert lib.kv_rope_turns(NULL, 1, out) == -1
    with pytest.raises(ValueError):
        binding.kv_rope_turns(torch.zeros(2, 2))


@pytest.mark.parametrize("freq", [1.0, -1.0, 0.1, 2.0 ** -40, -1e-7, 3.0, 6.283185307179586,
                                  -6.283185307179586, 1e4, 2.0 ** 30 - 1, 5e-324, 0.0]
                         + [10000.0 ** (-2 * i / 128) for i in range(64)])
def test_turns_are_right_to_the_last_places(lib, freq):
    """Within four units of 2^-64: a position may multiply the error by 2^31. The quotient's two
    parts are each cut once (two units), the second is off by a relative 2^-50 of at most 2^-53
    of the angle (under one unit up to 2^27 turns), and the 2 pi used here by 10^-60."""
    turn = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    got = binding.kv_rope_turns([freq]).item() % 2 ** 64
    want = Fraction(freq) / turn % 1 * 2 ** 64
    err = abs(got - want)
    assert min(err, 2 ** 64 - err) <= 4
