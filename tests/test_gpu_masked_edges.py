"""Windows and trees at their edges: waits that run out, lengths and offsets that are none, rows of
nobody, far pages, streams and graphs."""

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, f64, need_gpu
from test_gpu_masked_attn import Masked, bush, line
from test_gpu_prompt import Case, half_step
from test_gpu_prompt_edges import long_items

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


def masked(c, kind, **kw):
    """The call on a plain case: a window that reaches the first token, or a tree of one row."""
    if kind == "window":
        return skv.kv_window_attn(c.kv, c.q, c.scale, 2 ** 31 - 1, **kw)
    up = torch.full((c.q.shape[0],), -1, dtype=torch.int32, device="cuda")
    return skv.kv_tree_attn(c.kv, c.q, c.scale, up, **kw)


KINDS = ["window", "tree"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("shares", [1, 2])
def test_waits_that_run_out_are_flagged_and_end_the_call(wait_limit, kind, D, shares):
    """Without any patience every warp gives up, and the call says so and ends; the next one is as
    ever. A limit for copies does not end items of 40 ms. (Two shares: few rows.)"""
    c = long_items(D, 1 << 22, Hkv=8)
    ref, ref_lse = masked(c, kind, num_shares=shares)
    assert_no_device_error()
    for limit, want in ((0, (-6, 16)), (200_000, (0, 0)), (0, (-6, 16)), (2 ** 64 - 1, (0, 0))):
        wait_limit(limit)
        out, lse = masked(c, kind, num_shares=shares)
        wait_limit(2_000_000_000)
        assert skv.kv_check_device_errors() == want
        if want == (0, 0):
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,past,D,G,PS,shares", [
    ((700, 1, 129, 64), (0, 2000, 90, 33), 128, 4, 16, 0),
    ((700, 1, 129, 64), (0, 2000, 90, 33), 64, 1, 32, 1),
    ((1, 2, 1), (3000, 1234, 4001), 128, 8, 64, 7),
    ((1, 2, 1), (3000, 1234, 4001), 64, 2, 16, 0),
    ((5, 3, 4), (3000, 1234, 4001), 128, 4, 16, 0),
])
def test_under_any_wait_limit_the_bits_are_right_or_flagged(wait_limit, kind, new, past, D, G, PS,
                                                            shares):
    c = Masked(new, past, "bf16", D, G, PS=PS, tail=3, window=300 if kind == "window" else None,
               sinks=5, parents=[bush(n, 2 + n) for n in new] if kind == "tree" else None)
    if kind == "tree":
        c.up = torch.cat((c.up, c.up.new_zeros(3)))
    ref, ref_lse = c.attend(num_shares=shares)
    assert_no_device_error()
    for limit in (0, 1, 1000, 8000, 20000):
        for _ in range(4):
            out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
            lse = torch.full(c.q.shape[:2], -9.0, device="cuda")
            wait_limit(limit)
            c.attend(num_shares=shares, out=out, lse=lse)
            wait_limit(2_000_000_000)
            st, flags = skv.kv_check_device_errors()
            assert (st, flags) in ((0, 0), (-6, 16))
            if st == 0:
                assert torch.equal(out[:c.T], ref[:c.T]) and torch.equal(lse[:c.T], ref_lse[:c.T])
            assert (out[c.T:] == -9.0).all() and (lse[c.T:] == -9.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 2), ("bf16", 64, 8), ("fp32", 128, 2)])
@pytest.mark.parametrize("new", [(2, 3, 1), (40, 90, 33)])
def test_bad_lengths_and_offsets_leave_sequences_out(kind, dtype, D, G, new):
    c = Masked(new, (30, 40, 20), dtype, D, G, window=25 if kind == "window" else None, sinks=2,
               parents=[bush(n, n) for n in new] if kind == "tree" else None)
    ref, _, tol, _ = c.attn_bounds(c.q)
    kept = list(range(new[0])) + list(range(new[0] + new[1], c.T))
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, new[1] - 1):
        out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
        c.set_len([c.lens[0], bad, c.lens[2]])
        c.attend(out=out)
        assert skv.kv_check_device_errors() == (-5, 2)
        assert (out[new[0]:new[0] + new[1]] == 7.0).all()
        c.set_len(c.lens)
        assert (np.abs(f64(out) - ref) <= tol)[kept].all()
    for cu in ((0, 5, 2, 4), (3, 4, 5, 6), (0, -7, 2, 3), (0, 1, 2, c.T + 9)):
        c.attend(cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags & 2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,new", [("bf16", (2, 1)), ("bf16", (50, 70)), ("fp32", (2, 1)),
                                       ("fp32", (50, 70))])
def test_rows_of_nobody_and_no_rows(kind, dtype, new):
    c = Masked(new, (30, 400), dtype, tail=4, window=25 if kind == "window" else None,
               parents=[bush(n, n) for n in new] if kind == "tree" else None)
    if kind == "tree":
        c.up = torch.cat((c.up, c.up.new_full((4,), 10 ** 6)))
    out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], 7.0, device="cuda")
    c.q[c.T:] = float("nan")
    c.attend(out=out, lse=lse)
    assert_no_device_error()
    c.check_attn(c.q[:c.T], out[:c.T], lse[:c.T])
    assert (out[c.T:] == 7.0).all() and (lse[c.T:] == 7.0).all()
    out.fill_(7.0)
    c.attend(out=out, lse=lse, cu_tokens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert_no_device_error()
    assert (out == 7.0).all()
    if kind == "window":
        e, _ = skv.kv_window_attn(c.kv, c.q[:0], c.scale, 5, cu_tokens=c.cu * 0)
        assert e.shape[0] == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 128)])
@pytest.mark.parametrize("new", [(2, 1), (100, 77)])
def test_pages_past_32_bit_offsets(kind, dtype, D, new):
    """The last pages of pools of more than 2^31 elements."""
    c = Masked(new, (300, 40), dtype, D, G=4, extra=0, window=90 if kind == "window" else None,
               sinks=3, parents=[bush(n, n) for n in new] if kind == "tree" else None)
    ref, ref_lse = c.attend()
    need = c.k_pool.shape[0]
    NP = 2 ** 31 // (2 * 16 * D) + 40
    k = torch.zeros((NP, 2, 16, D), dtype=c.k_pool.dtype, device="cuda")
    v = torch.zeros_like(k)
    k[-need:], v[-need:] = c.k_pool, c.v_pool
    table = torch.where(c.table >= 0, c.table + (NP - need), c.table).to(torch.int32)
    c.kv = skv.PagedKV(k, v, table, c.seq_lens)
    out, lse = c.attend()
    assert_no_device_error()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [(1, 2, 1), (5, 8, 4), (60, 90, 33)])
def test_two_captured_calls_with_a_workspace_each_at_once(kind, new):
    """Graphs replayed on two streams at the same time, and the same bits every time."""
    cs = [Masked(new, (900, 4000, 77), seed=s, window=300 if kind == "window" else None, sinks=4,
                 parents=[bush(n, n + s) for n in new] if kind == "tree" else None)
          for s in (1, 2)]
    refs, graphs, outs, keep = [], [], [], []
    for c in cs:
        ws = torch.empty((skv.kv_prefill_attn_workspace_size(c.kv, c.Hq, c.T),),
                         dtype=torch.uint8, device="cuda")
        out = torch.empty((c.T, c.Hq, c.D), dtype=c.q.dtype, device="cuda")
        lse = torch.empty((c.T, c.Hq), device="cuda")
        refs.append(c.attend())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.attend(workspace=ws, out=out, lse=lse)
        graphs.append(graph)
        outs.append((out, lse))
        keep.append(ws)
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for out, lse in outs:
            out.fill_(-3.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (out, lse), (ref, ref_lse) in zip(outs, refs):
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert_no_device_error()


def test_single_rows_of_a_line_equal_the_prompt_attention_to_rounding():
    """Drafts in one line through both calls: the same rows by kernels of their own."""
    c = Masked((4, 4), (2500, 63), G=4, parents=[line(4)] * 2)
    for out, lse in (c.attend(), skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)):
        assert_no_device_error()
        c.check_attn(c.q, out, lse)


def test_calls_that_the_binding_refuses():
    c = Masked((3, 2), (9, 9), window=4)
    for name, fn in (("window", lambda **k: skv.kv_window_attn(c.kv, c.q, c.scale, 4, **k)),
                     ("tree", lambda **k: skv.kv_tree_attn(
                         c.kv, c.q, c.scale, torch.zeros(5, dtype=torch.int32, device="cuda"),
                         **k))):
        with pytest.raises(ValueError):
            fn()                                                   # one row per sequence
        with pytest.raises(ValueError):
            fn(cu_tokens=c.cu.cpu())
        with pytest.raises(ValueError):
            fn(cu_tokens=c.cu.long())
        with pytest.raises(ValueError):
            fn(cu_tokens=c.cu, out=torch.empty((5, 8, 64), device="cuda"))
        with pytest.raises(binding.KVError):
            fn(cu_tokens=c.cu, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    for bad in (torch.zeros(4, dtype=torch.int32, device="cuda"),
                torch.zeros(5, dtype=torch.int64, device="cuda"), torch.zeros(5, dtype=torch.int32),
                torch.zeros(10, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            skv.kv_tree_attn(c.kv, c.q, c.scale, bad, cu_tokens=c.cu)
    for window, sinks in ((0, 0), (-1, 0), (3, -1)):
        with pytest.raises(binding.KVError):
            skv.kv_window_attn(c.kv, c.q, c.scale, window, sinks, cu_tokens=c.cu)
    p = Case((3, 2), (9, 9))
    refs = torch.zeros(p.k_pool.shape[0], dtype=torch.int32, device="cuda")
    lens = torch.tensor([12, 11], dtype=torch.int32, device="cuda")
    for bad in (dict(refs=refs[:-1]), dict(refs=refs.long()), dict(new_lens=lens[:1]),
                dict(new_lens=lens.view(1, 2)), dict(keep_lens=lens[:1]), dict(parents=lens[:1]),
                dict(parents=lens, table=p.table), dict(table=p.table[:1]),
                dict(copies=torch.zeros((2, 3), dtype=torch.int32, device="cuda"))):
        args = {"refs": refs, "new_lens": lens, **bad}
        with pytest.raises((ValueError, binding.KVError)):
            skv.kv_update_pages(p.kv, args.pop("refs"), args.pop("new_lens"), **args)
    keep = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for bad in (dict(keep=keep[0]), dict(keep=keep[:, :0]), dict(keep_cnt=lens[:1]),
                dict(keep=keep[:1]), dict(stats=torch.zeros(3, device="cuda")),
                dict(new_lens=p.seq_lens)):
        args = {"keep": keep, "keep_cnt": lens * 0, **bad}
        with pytest.raises((ValueError, binding.KVError)):
            skv.kv_compact(p.kv, args.pop("keep"), args.pop("keep_cnt"), cu_tokens=p.cu, **args)
    for pairs in (keep, keep[0], keep[:, :2].contiguous().long()):
        with pytest.raises(ValueError):
            skv.kv_copy_pages(p.kv, pairs)
    assert_no_device_error()


@pytest.mark.parametrize("dtype,D,G,n", [("bf16", 128, 4, 1), ("bf16", 64, 8, 300),
                                         ("bf16", 128, 8, 3), ("fp32", 64, 2, 1),
                                         ("fp32", 128, 2, 100)])
@pytest.mark.parametrize("window,sinks", [(700, 5), (1, 0), (64, 130)])
def test_windows_at_the_end_of_the_longest_tables(dtype, D, G, n, window, sinks):
    """Rows at positions near 2^31: the same tokens in a short table give the same rows."""
    PS, stride = 64, (2 ** 31 - 1 - 256) // 64
    length = stride * PS - 5
    keep = -(-sinks // PS) + (window + n) // PS + 3            # pages that rows may see
    c = Case((n,), (PS * keep,), dtype, D, G, PS=PS, extra=0)
    first = -(-sinks // PS)                                    # pages with sinks
    tail = keep - first
    # the short sequence: the sinks' pages, then the long one's last pages
    short_len = (first + tail) * PS - 5
    pages = c.table[0, :keep]
    c.kv = skv.PagedKV(c.k_pool, c.v_pool, pages.view(1, -1).contiguous(),
                       torch.tensor([short_len], dtype=torch.int32, device="cuda"))
    ref, ref_lse = skv.kv_window_attn(c.kv, c.q, c.scale, window, sinks, cu_tokens=c.cu)
    table = torch.full((1, stride), -1, dtype=torch.int32, device="cuda")
    table[0, :first] = pages[:first]
    table[0, stride - tail:] = pages[first:]
    kv = skv.PagedKV(c.k_pool, c.v_pool, table,
                     torch.tensor([length], dtype=torch.int32, device="cuda"))
    out, lse = skv.kv_window_attn(kv, c.q, c.scale, window, sinks, cu_tokens=c.cu)
    assert_no_device_error()
    # The same scores, cut into other tiles: sums of at most 1024 terms in another order (2^-13 of
    # them), and per side the rounding of the probabilities (bf16) and of the output.
    most = 1.01 * c.v_pool.abs().float().max().item()
    rel = 2.0 ** -13 + 4 * half_step(dtype)
    assert np.abs(f64(out) - f64(ref)).max() <= rel * most
    assert (np.abs(f64(lse) - f64(ref_lse)) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(f64(ref_lse))).all()
