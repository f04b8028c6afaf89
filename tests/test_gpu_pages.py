"""Compaction, page copies and page tables against an oracle that goes token by token. Everything
here moves values or counts them: results are equal, not near."""

import random

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import pages as oracle

from gpu_helpers import assert_no_device_error, f32, need_gpu
from test_gpu_prompt import DT, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def lists(kept, extra=0):
    """keep (rows padded with an index that is never read) and keep_cnt."""
    most = max(1, max(map(len, kept))) + extra
    return ints([k + [-77] * (most - len(k)) for k in kept]), ints([len(k) for k in kept])


def all_stats(c, seed=3):
    """Statistics with a value of their own in every entry, so that any write shows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (c.k_pool.shape[0], c.Hkv, 2, c.D)
    return torch.randn(shape, generator=gen, device="cuda").to(DT[c.dtype])


def check_compact(c, kept, counts=None, stats=None, **kw):
    counts = c.new if counts is None else counts
    k0, v0 = f32(c.k_pool), f32(c.v_pool)
    stats = all_stats(c) if stats is None else stats
    s0 = stats.clone()
    keep, cnt = lists(kept)
    lens = skv.kv_compact(c.kv, keep, cnt, stats, **{"cu_tokens": c.cu, **kw})
    assert_no_device_error()
    table = c.table.cpu().numpy()
    k, v, ref_lens, touched = oracle.compact(k0, v0, table, c.lens, counts, kept, c.PS)
    assert lens.tolist() == ref_lens
    assert np.array_equal(f32(c.k_pool), k, equal_nan=True)
    assert np.array_equal(f32(c.v_pool), v, equal_nan=True)
    assert c.seq_lens.tolist() == c.lens             # the caller's to replace
    # statistics: the full build's at the new lengths where tokens may have gone, else untouched
    c.set_len(ref_lens)
    built = skv.kv_build_page_stats(c.kv, stats=s0.clone())
    c.set_len(c.lens)
    for b, p in touched:
        s0[table[b, p]] = built[table[b, p]]
    assert np.array_equal(f32(stats), f32(s0), equal_nan=True)
    return lens


def some(rng, n, most):
    return sorted(rng.sample(range(n), min(n, rng.randrange(most + 1))))


COMPACT = [
    # candidates, tokens before, dtype, D, Hkv, PS
    ((8,), (0,), "bf16", 128, 2, 16),
    ((26, 1, 0, 64, 9), (500, 16, 40, 63, 7), "bf16", 128, 8, 16),
    ((26, 1, 0, 64, 9), (500, 16, 40, 63, 7), "bf16", 64, 1, 64),
    ((33, 130), (77, 0), "fp32", 128, 2, 32),
    ((33, 130), (77, 0), "fp32", 64, 16, 16),
    (tuple((5 * i) % 13 for i in range(60)), tuple((11 * i) % 70 for i in range(60)), "bf16", 64,
     2, 32),
]


@pytest.mark.parametrize("new,past,dtype,D,Hkv,PS", COMPACT)
@pytest.mark.parametrize("seed", [1, 2])
def test_compact(new, past, dtype, D, Hkv, PS, seed):
    rng = random.Random(seed)
    c = Case(new, past, dtype, D, 1, Hkv, PS, seed=seed)
    check_compact(c, [some(rng, n, 9) for n in new])


@pytest.mark.parametrize("which", ["none", "all", "first", "last", "odd", "tail"])
@pytest.mark.parametrize("past", [0, 16, 21])
def test_compact_of_particular_lists(which, past):
    n = 70
    kept = {"none": [], "all": list(range(n)), "first": list(range(20)), "last": [n - 1],
            "odd": list(range(1, n, 2)), "tail": list(range(40, n))}[which]
    check_compact(Case((n, 3), (past, 5), G=1), [kept, [0, 2]])


@pytest.mark.parametrize("dtype,D,Hkv,PS,n", [("bf16", 128, 2, 16, 9000), ("bf16", 64, 1, 64, 5001),
                                              ("fp32", 128, 8, 32, 3333), ("fp32", 64, 2, 16, 1030),
                                              ("bf16", 128, 1, 16, 20011)])
@pytest.mark.parametrize("how", ["eighth", "half", "all but some", "shifted"])
def test_compact_of_whole_sequences(dtype, D, Hkv, PS, n, how):
    """Every token is a candidate: an eviction, in many batches of a block."""
    rng = random.Random(n)
    c = Case((n, 40), (0, 0), dtype, D, 1, Hkv, PS)
    kept = {"eighth": sorted(rng.sample(range(n), n // 8)),
            "half": sorted(rng.sample(range(n), n // 2)),
            "all but some": [i for i in range(n) if i % 997 != 5],
            "shifted": list(range(1, n))}[how]
    check_compact(c, [kept, [0, 39]], counts=c.lens, cu_tokens=None)


def test_compact_keeps_the_full_builds_rule_for_nan():
    """A NaN of a page's first key stays, one of a later key does not count."""
    c = Case((60, 60), (3, 0), G=1)
    for t in (1, 20, 33):
        c.k_pool[c.table[0, t // 16].long(), :, t % 16, :5] = float("nan")
        c.k_pool[c.table[1, t // 16].long(), :, t % 16, 7:9] = float("nan")
    check_compact(c, [[5, 13, 14, 17, 30, 41, 42, 43, 44, 45, 46, 47, 48, 49, 50, 51, 52, 53],
                      list(range(1, 40, 3))])


def test_compact_without_statistics_and_into_given_lengths():
    c = Case((20,), (30,), G=1)
    keep, cnt = lists([[2, 3, 9]], extra=4)
    k0 = f32(c.k_pool)
    lens = ints([0])
    assert skv.kv_compact(c.kv, keep, cnt, cu_tokens=c.cu, new_lens=lens) is lens
    assert_no_device_error()
    k, *_ = oracle.compact(k0, k0, c.table.cpu().numpy(), c.lens, c.new, [[2, 3, 9]], 16)
    assert np.array_equal(f32(c.k_pool), k) and lens.tolist() == [33]


def test_compact_flags_what_does_not_fit():
    """Counts and indices that are none; the other sequences are compacted all the same."""
    for bad, flags in (([1, 25], 4), ([3, 2], 4), ([4, 4], 4), ([-1], 4), ([2 ** 31 - 1], 4)):
        c = Case((20, 20), (30, 10), G=1)
        stats = all_stats(c)
        keep, cnt = lists([bad, [1, 5]])
        k0 = f32(c.k_pool)
        skv.kv_compact(c.kv, keep, cnt, stats, cu_tokens=c.cu)
        assert skv.kv_check_device_errors() == (-5, flags)
        own = c.table[1].long().cpu().numpy()
        k, *_ = oracle.compact(k0, k0, c.table.cpu().numpy(), c.lens, c.new, [[], [1, 5]], 16)
        used = own[own >= 0]
        assert np.array_equal(f32(c.k_pool)[used], k[used])
    for count in (-1, 21, 3):                        # 3: more than the list holds
        c = Case((20, 20), (30, 10), G=1)
        stats, keep, cnt = all_stats(c), *lists([[1, 2], [0, 5]])
        cnt[0] = count
        before = (c.k_pool.clone(), c.v_pool.clone(), stats.clone())
        lens = skv.kv_compact(c.kv, keep, cnt, stats, cu_tokens=c.cu)
        assert skv.kv_check_device_errors() == (-5, 4)
        assert lens.tolist() == [50, 12]
        own = c.table[0].long()
        own = own[own >= 0]
        assert torch.equal(c.k_pool[own], before[0][own])
        assert torch.equal(c.v_pool[own], before[1][own])
        assert torch.equal(stats[own], before[2][own])


def test_compact_flags_bad_lengths_offsets_and_pages():
    c = Case((20, 20), (30, 10), G=1)
    keep, cnt = lists([[1, 2], [0, 5]])
    c.set_len([10 ** 6, 30])
    lens = skv.kv_compact(c.kv, keep, cnt, cu_tokens=c.cu)
    status, flags = skv.kv_check_device_errors()
    assert status == -5 and flags & 2 and lens.tolist() == [0, 12]
    c = Case((20, 20), (30, 10), G=1)
    lens = skv.kv_compact(c.kv, keep, cnt, cu_tokens=ints([0, 60, 40]))
    status, flags = skv.kv_check_device_errors()
    assert status == -5 and flags & 2 and lens.tolist() == [50, 30]
    c = Case((20, 20), (30, 10), G=1)
    c.table[0, 1] = -1
    k0 = f32(c.k_pool)
    skv.kv_compact(c.kv, keep, cnt, cu_tokens=c.cu)
    assert skv.kv_check_device_errors() == (-5, 1)
    rest = sorted(set(range(k0.shape[0])) - set(c.table[1].tolist()))
    assert np.array_equal(f32(c.k_pool)[rest], k0[rest])


def test_compact_past_32_bit_offsets():
    NP = 2 ** 31 // (2 * 16 * 128) + 40
    c = Case((90, 5), (5, 16), G=1, extra=0)
    need, small_k, small_v, table = c.k_pool.shape[0], c.k_pool, c.v_pool, c.table.clone()
    big_k = torch.empty((NP, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    big_k[-need:], big_v[-need:] = small_k, small_v
    stats = torch.zeros((NP, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    big = skv.PagedKV(big_k, big_v, torch.where(table >= 0, table + (NP - need), table).to(
        torch.int32), c.seq_lens)
    kept = [list(range(0, 90, 2)), [1, 4]]
    keep, cnt = lists(kept)
    skv.kv_compact(big, keep, cnt, stats, cu_tokens=c.cu)
    skv.kv_copy_pages(big, ints([[NP - 1, 0], [1, NP - 2]]), stats)
    assert_no_device_error()
    before = big_k[0].clone(), stats[0].clone()
    small = torch.zeros((need, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    skv.kv_compact(c.kv, keep, cnt, small, cu_tokens=c.cu)
    assert torch.equal(before[0], small_k[-1]) and torch.equal(before[1], small[-1])
    assert torch.equal(big_k[-need:-2], small_k[:-2]) and torch.equal(big_v[-need:-2], small_v[:-2])
    assert torch.equal(stats[-need:-2], small[:-2])


# ------------------------------------------------------------------------- page copies

@pytest.mark.parametrize("dtype,D,Hkv,PS", [("bf16", 128, 8, 16), ("bf16", 64, 1, 16),
                                            ("fp32", 128, 3, 64), ("fp32", 64, 16, 32)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_copy_pages(dtype, D, Hkv, PS, n):
    c = Case((5,), (0,), dtype, D, 1, Hkv, PS, extra=2 * n + 9)
    stats = all_stats(c)
    order = torch.randperm(c.k_pool.shape[0], device="cuda")[:2 * n].to(torch.int32)
    pairs = order.view(n, 2).contiguous()
    ref = [x.clone() for x in (c.k_pool, c.v_pool, stats)]
    skip = list(range(0, n, 3)) if n > 1 else []
    for i in skip:
        pairs[i, i % 2] = -1 - i
    live = [i for i in range(n) if i not in skip]
    for x in ref:
        x[pairs[live, 1].long()] = x[pairs[live, 0].long()]
    bare = stats.clone()
    skv.kv_copy_pages(c.kv, pairs, stats)
    assert_no_device_error()
    for x, y in zip((c.k_pool, c.v_pool, stats), ref):
        assert torch.equal(x, y)
    stats.copy_(bare)
    skv.kv_copy_pages(c.kv, pairs)                   # without statistics
    assert torch.equal(stats, bare)
    skv.kv_copy_pages(c.kv, pairs[:0])
    assert_no_device_error()


def test_copy_pages_beyond_the_pool_are_flagged():
    c = Case((5,), (0,), extra=9)
    NP = c.k_pool.shape[0]
    before = c.k_pool.clone()
    skv.kv_copy_pages(c.kv, ints([[0, NP], [NP + 5, 1], [2, 3]]), all_stats(c))
    assert skv.kv_check_device_errors() == (-5, 1)
    before[3] = before[2]
    assert torch.equal(c.k_pool, before)


# ------------------------------------------------------------------------- page tables

class Pool:
    """A pool's counts and a batch's page table, here and in the oracle."""

    def __init__(self, pages, stride, PS=16):
        self.NP, self.stride, self.PS = pages, stride, PS
        self.k = torch.empty((pages, 1, PS, 64), dtype=torch.bfloat16, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = np.full((1, stride), -1, dtype=np.int64)
        self.lens = [0]
        self.kv = skv.PagedKV(self.k, self.k, ints(self.table.tolist()), ints(self.lens))

    def step(self, want, keep=None, parents=None, window=0, sinks=0, flags=0, **kw):
        """One call, compared with the oracle; the batch moves on to its result."""
        rows = len(want)
        ref = oracle.update_pages(self.table, self.lens, self.refs.tolist(), rows, parents,
                                  self.lens if keep is None else keep, want, self.PS, window,
                                  sinks)
        table, copies, left = skv.kv_update_pages(
            self.kv, self.refs, ints(want), keep_lens=None if keep is None else ints(keep),
            parents=None if parents is None else ints(parents), window=window, sinks=sinks, **kw)
        st, got = skv.kv_check_device_errors()
        assert got == flags and (st == 0) == (flags == 0)
        assert np.array_equal(table.cpu().numpy(), ref[0])
        assert self.refs.tolist() == ref[1]
        assert np.array_equal(copies.cpu().numpy(), ref[2])
        assert left.tolist() == [ref[3]]
        self.table = ref[0]
        if ref[3] >= 0:
            self.lens = list(want)
        else:
            self.lens = list(keep) if keep is not None else self.lens
        self.kv = skv.PagedKV(self.k, self.k, table, ints(self.lens))
        return ref

    def check_counts(self):
        used = self.table[self.table >= 0]
        assert np.array_equal(np.bincount(used, minlength=self.NP), self.refs.cpu().numpy())


def test_sequences_come_grow_fork_and_go():
    p = Pool(200, 40)
    p.step([100, 17, 0, 16], parents=[-1] * 4, keep=[0] * 4)      # four new sequences
    p.step([101, 18, 1, 17])                                       # a token each, in place
    p.step([130, 130, 131, 1, 18], parents=[0, 0, 0, 2, 3], keep=[101, 101, 101, 1, 17])
    p.check_counts()
    p.step([130, 130, 131, 1, 18])                                 # nothing to do
    p.step([120, 140, 30, 2, 18], keep=[110, 128, 16, 0, 18])      # tokens dropped, then others
    p.check_counts()
    p.step([50], parents=[1], keep=[37])                           # the others go
    p.check_counts()
    p.step([0], keep=[0])
    assert p.refs.sum() == 0


def test_partial_pages_are_kept_by_their_last_holder():
    """Rows that alone share a page: the last keeps it. Held elsewhere too: all copy."""
    p = Pool(64, 8)
    p.step([21], parents=[-1], keep=[0])
    ref = p.step([22, 21, 25], parents=[0, 0, 0], keep=[21, 21, 21])      # row 1 does not grow
    assert (ref[2] >= 0).all(1).tolist() == [True, False, True]
    p = Pool(64, 8)
    p.step([21], parents=[-1], keep=[0])
    ref = p.step([22, 22, 25], parents=[0, 0, 0], keep=[21, 21, 21])
    assert (ref[2] >= 0).all(1).tolist() == [True, True, False]
    p = Pool(64, 8)
    p.step([21], parents=[-1], keep=[0])
    p.refs[p.table[0, 1]] += 1                                     # a prefix cache holds it
    p.step([22, 22], parents=[0, 0], keep=[21, 21])
    p = Pool(64, 8)                                                # shared full pages need no copy
    p.step([32], parents=[-1], keep=[0])
    ref = p.step([33, 34], parents=[0, 0], keep=[32, 32])
    assert (ref[2] == -1).all()
    ref = p.step([33, 34], keep=[30, 30])                          # now a partial page again
    assert (ref[2] >= 0).all(1).tolist() == [True, False]
    p.check_counts()


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (40, 0), (40, 33), (1000, 4)])
def test_windows_give_pages_back(window, sinks):
    p = Pool(400, 40, PS=16)
    p.step([300, 15, 16, 17], parents=[-1] * 4, keep=[0] * 4)
    for n in range(40):
        p.step([x + 1 + n % 3 for x in p.lens], window=window, sinks=sinks)
        p.check_counts()


def test_what_a_window_gives_back_is_never_read_again():
    """The pages that stay hold every token that the next rows see."""
    p = Pool(400, 40)
    p.step([333], parents=[-1], keep=[0])
    for window, sinks in ((300, 20), (100, 17), (33, 4), (16, 4), (15, 1), (1, 0)):
        p.step([p.lens[0] + 1], window=window, sinks=sinks)
        pos = p.lens[0] - 1
        seen = {u // 16 for u in range(pos + 1) if u > pos - window or u < sinks}
        assert all(p.table[0, q] >= 0 for q in seen)


def test_too_few_pages_leave_rows_as_they_were():
    p = Pool(10, 16)
    p.step([100, 30], parents=[-1, -1], keep=[0, 0])               # 7 + 2 of 10
    ref = p.step([101, 60, 31], parents=[0, 1, 1], keep=[100, 30, 30], flags=32)
    assert ref[3] == -2                                            # a copy and two pages, one left
    p.check_counts()
    p.step([112, 31], parents=[0, 1], keep=[100, 30])              # without the fork it fits
    p.check_counts()
    p.step([16 * 10, 0], parents=[0, -1], keep=[100, 0])           # all there are
    assert (p.refs == 1).all()


@pytest.mark.parametrize("pages,stride,PS", [(1000, 30, 16), (5003, 130, 64), (129, 9, 32),
                                             (70001, 1100, 16)])
def test_random_steps(pages, stride, PS):
    rng = random.Random(pages)
    p = Pool(pages, stride, PS)
    fails = 0
    for n in range(25):
        rows = rng.choice((1, 3, 17, 60))
        parents = None if rng.random() < 0.4 else \
            [rng.randrange(-1, len(p.lens)) for _ in range(rows)]
        old = p.lens if parents is None else [p.lens[q] if q >= 0 else 0 for q in parents]
        keep = [max(0, x - rng.choice((0, 0, 1, 5, 100))) for x in old]
        most = min(stride * PS, 2 * pages * PS // max(1, len(old)))
        want = [min(stride * PS, max(k, min(most, k + rng.choice((0, 1, 1, 7, 200, most)))))
                for k in keep]
        window, sinks = rng.choice(((0, 0), (0, 0), (50, 4), (300, 0)))
        args = (p.table, p.lens, p.refs.tolist(), len(want), parents, keep, want, PS, window, sinks)
        short = oracle.update_pages(*args)[3] < 0
        fails += short
        p.step(want, keep=keep, parents=parents, window=window, sinks=sinks,
               flags=32 if short else 0)
        p.check_counts()
    assert fails < 25


def test_many_rows():
    """More rows than the cluster has threads, most of them forks of a few."""
    p = Pool(40000, 12)
    p.step([20, 33, 48], parents=[-1] * 3, keep=[0] * 3)
    rows = 9001
    parents = [i % 3 for i in range(rows)]
    p.step([(20, 33, 48)[q] + i % 2 for i, q in enumerate(parents)], parents=parents,
           keep=[(20, 33, 48)[q] for q in parents])
    p.check_counts()
    p.step([n + 1 for n in p.lens])
    p.check_counts()


def test_pages_are_lists_of_pool_and_other_holders():
    """Pages that a holder outside the table counts are not handed out; a table of its own."""
    p = Pool(50, 10)
    p.refs[:20:2] = 1
    p.step([100], parents=[-1], keep=[0])
    assert p.table[0, :7].tolist() == [1, 3, 5, 7, 9, 11, 13]
    out = torch.full((1, 10), 99, dtype=torch.int32, device="cuda")
    p.step([120], table=out, copies=torch.zeros((1, 2), dtype=torch.int32, device="cuda"),
           free_left=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert p.kv.page_table is out


def test_numbers_that_do_not_fit_are_flagged():
    def case():
        p = Pool(50, 10)
        p.step([40, 50], parents=[-1, -1], keep=[0, 0])
        return p

    for keep, want, parents, flags, lens in (
            ([41, 50], [45, 51], None, 2, [40, 51]),          # keep beyond the tokens held
            ([-1, 50], [45, 51], None, 2, [40, 51]),
            ([40, 50], [39, 51], None, 2, [40, 51]),          # fewer wanted than kept
            ([40, 50], [161, 51], None, 2, [40, 51]),         # more than a table row
            ([40, 50], [41, 51], [0, 2], 6, None),            # no such row: a new one, of 0 tokens
            ([40, 0], [41, 0], [0, -2], 4, None)):
        p = case()
        if lens is None:
            good_parents, good_keep, good_want = [0, -1], [40, 0], [41, 0]
        else:
            good_parents, good_keep, good_want = parents, [40, 50], lens
        ref = oracle.update_pages(p.table, p.lens, p.refs.tolist(), 2, good_parents, good_keep,
                                  good_want, 16)
        table, copies, left = skv.kv_update_pages(
            p.kv, p.refs, ints(want), keep_lens=ints(keep),
            parents=None if parents is None else ints(parents))
        assert skv.kv_check_device_errors() == (-5, flags)
        assert np.array_equal(table.cpu().numpy(), ref[0]) and p.refs.tolist() == ref[1]
        assert left.tolist() == [ref[3]]
    p = case()
    p.kv.page_table[0, 1], p.kv.page_table[0, 5] = 50, -2     # no pages: taken as unmapped
    held = p.table[0, 1]
    table, _, _ = skv.kv_update_pages(p.kv, p.refs, ints([40, 50]))
    assert skv.kv_check_device_errors() == (-5, 1)
    assert table[0, 1] == -1 and (table[0, 3:] == -1).all() and p.refs[held] == 1


def test_captured_update_follows_its_inputs():
    p = Pool(300, 20)
    p.step([50, 70], parents=[-1, -1], keep=[0, 0])
    want, keep, parents = ints([51, 71]), ints([50, 70]), ints([0, 1])
    table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    copies = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    left = torch.empty(1, dtype=torch.int32, device="cuda")
    refs0 = p.refs.clone()
    args = dict(keep_lens=keep, parents=parents, table=table, copies=copies, free_left=left)
    skv.kv_update_pages(p.kv, p.refs, want, **args)
    p.refs.copy_(refs0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skv.kv_update_pages(p.kv, p.refs, want, **args)
    want.copy_(ints([90, 66]))
    keep.copy_(ints([60, 60]))
    parents.copy_(ints([1, 1]))
    ref = oracle.update_pages(p.table, p.lens, refs0.tolist(), 2, [1, 1], [60, 60], [90, 66], 16)
    graph.replay()
    assert_no_device_error()
    assert np.array_equal(table.cpu().numpy(), ref[0]) and p.refs.tolist() == ref[1]
    assert np.array_equal(copies.cpu().numpy(), ref[2]) and left.tolist() == [ref[3]]


def test_calls_on_a_stream_given_by_argument():
    """A call's own buffers are the stream's: not ones that the current stream still writes to."""
    s = torch.cuda.Stream()
    for _ in range(5):
        p = Pool(300, 20)
        p.step([50, 70], parents=[-1, -1], keep=[0, 0])
        want, keep, parents = ints([51, 75]), ints([50, 50]), ints([0, 0])
        ref = oracle.update_pages(p.table, p.lens, p.refs.tolist(), 2, [0, 0], [50, 50], [51, 75],
                                  16)
        c = Case((20, 30), (30, 7), G=1)
        kept, k0 = [[1, 4], [0, 2, 29]], f32(c.k_pool)
        lists_ = lists(kept)
        old = [torch.empty(x, dtype=torch.int32, device="cuda")
               for x in ((2, 20), (2, 2), (1,), (2,))]
        torch.cuda.synchronize()
        torch.cuda._sleep(10_000_000)
        for x in old:                          # freed with a write of this stream still to come
            x.fill_(-9)
        del old, x
        table, copies, left = skv.kv_update_pages(p.kv, p.refs, want, keep_lens=keep,
                                                  parents=parents, stream=s)
        lens = skv.kv_compact(c.kv, *lists_, cu_tokens=c.cu, stream=s)
        skv.kv_copy_pages(c.kv, ints([[-1, -1]]), stream=s)
        torch.cuda.synchronize()
        assert_no_device_error()
        assert np.array_equal(table.cpu().numpy(), ref[0]) and p.refs.tolist() == ref[1]
        assert np.array_equal(copies.cpu().numpy(), ref[2]) and left.tolist() == [ref[3]]
        k, _, ref_lens, _ = oracle.compact(k0, k0, c.table.cpu().numpy(), c.lens, c.new, kept, 16)
        assert np.array_equal(f32(c.k_pool), k) and lens.tolist() == ref_lens


def test_copies_of_many_pages():
    c = Case((5,), (0,), "bf16", 64, 1, 1, 16, extra=160_000)
    stats = all_stats(c)
    pairs = torch.randperm(c.k_pool.shape[0], device="cuda")[:140_000].to(torch.int32).view(-1, 2)
    ref = [x.clone() for x in (c.k_pool, c.v_pool, stats)]
    for x in ref:
        x[pairs[:, 1].long()] = x[pairs[:, 0].long()]
    skv.kv_copy_pages(c.kv, pairs.contiguous(), stats)
    assert_no_device_error()
    for x, y in zip((c.k_pool, c.v_pool, stats), ref):
        assert torch.equal(x, y)


def test_long_rows_of_a_table():
    """Two sequences of a few pages in rows of a million entries, one of which moves to its end."""
    p = Pool(100, 1 << 20)
    p.step([40, 100], parents=[-1, -1], keep=[0, 0])
    p.step([41, 101, 100], parents=[1, 1, 0], keep=[41, 100, 40])
    p.check_counts()
