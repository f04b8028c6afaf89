"""Attention within a sliding window and of drafted trees, against the float64 oracle; the error
bounds are those of causal attention (test_gpu_prompt.py), whose arithmetic the calls share."""

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import prompt
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, f64, need_gpu
from test_gpu_prompt import Case, half_step, spoil_the_rest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


class Masked(Case):
    """A cache and packed rows with a mask; the oracle reads the pools as they were made."""

    def __init__(self, *args, window=None, sinks=0, parents=None, **kw):
        super().__init__(*args, **kw)
        self.window, self.sinks, self.parents = window, sinks, parents
        self.clean = (f64(self.k_pool), f64(self.v_pool), self.table.cpu().numpy().copy())
        self.up = None if parents is None else torch.tensor(
            [p for t in parents for p in t], dtype=torch.int32, device="cuda")

    def give_back(self):
        """Unmaps the pages that no row sees, and leaves NaN and infinities in them."""
        for b, past in enumerate(self.past):
            for p in range(-(-self.lens[b] // self.PS)):
                if (p * self.PS >= self.sinks and
                        (p + 1) * self.PS <= past - self.window + 1 and self.new[b]):
                    P = int(self.table[b, p])
                    self.k_pool[P], self.v_pool[P] = float("nan"), float("inf")
                    self.table[b, p] = -1

    def hidden(self, b, n, length):
        if self.parents is not None:
            return prompt.tree_hidden(self.parents[b], length)
        return prompt.window_hidden(n, length, self.window, self.sinks)

    def attn_bounds(self, q):
        k, v, table = self.clean
        out, lse, mass, logit = prompt.prefill(f64(q), k, v, table, self.lens, self.cu_h, self.PS,
                                               self.scale, hidden_of=self.hidden)
        L = max(self.lens)
        rel = 2 * self.D * 2.0 ** -23 * logit + 2.0 ** -21 + L * 2.0 ** -23
        p = half_step("bf16") if self.dtype == "bf16" else 0.0
        tol = (rel + p)[..., None] * mass * 1.01 + half_step(self.dtype) * np.abs(out) * 1.01
        return out, lse, tol + 1e-30, rel + 2.0 ** -23 * np.abs(lse)

    def attend(self, **kw):
        kw.setdefault("cu_tokens", self.cu)
        if self.parents is not None:
            return skv.kv_tree_attn(self.kv, self.q, self.scale, self.up, **kw)
        return skv.kv_window_attn(self.kv, self.q, self.scale, self.window, self.sinks, **kw)


# --------------------------------------------------------------------------- windows

WINDOW = [
    # new, past, dtype, D, G, PS, shares, window, sinks
    ((1,), (0,), "bf16", 128, 4, 16, 0, 1, 0),
    ((1,), (3000,), "bf16", 128, 4, 16, 0, 1, 0),
    ((1,), (3000,), "bf16", 128, 8, 64, 0, 257, 4),
    ((300,), (0,), "bf16", 128, 4, 16, 1, 1, 0),
    ((300,), (0,), "bf16", 128, 4, 16, 0, 64, 4),
    ((700,), (1000,), "bf16", 128, 4, 16, 0, 200, 5),
    ((700,), (1000,), "bf16", 128, 1, 64, 3, 129, 200),
    ((700,), (1000,), "bf16", 64, 8, 32, 1, 128, 128),
    ((700,), (1000,), "bf16", 64, 2, 16, 29, 500, 1),
    ((40, 700, 0, 1, 130), (2000, 3, 7, 900, 128), "bf16", 128, 8, 32, 0, 300, 17),
    ((40, 700, 0, 1, 130), (2000, 3, 7, 900, 128), "bf16", 64, 1, 16, 7, 90, 0),
    ((1, 1, 1, 1), (0, 127, 5128, 900), "bf16", 128, 8, 16, 4, 128, 4),
    ((5, 5, 5), (4063, 1500, 700), "bf16", 64, 1, 16, 7, 1000, 130),
    ((5, 5, 5), (4063, 1500, 700), "bf16", 128, 2, 16, 0, 1000, 4064),
    ((900,), (200,), "bf16", 128, 4, 16, 0, 2 ** 31 - 1, 2 ** 31 - 1),
    ((900,), (200,), "bf16", 128, 4, 16, 0, 7, 2 ** 31 - 1),
    ((65, 1, 200), (0, 900, 64), "fp32", 64, 4, 16, 1, 50, 3),
    ((65, 1, 200), (0, 900, 64), "fp32", 128, 8, 64, 3, 64, 65),
    ((65, 1, 200), (1000, 900, 640), "fp32", 128, 8, 16, 0, 301, 20),
    ((1, 1, 1), (0, 700, 15), "fp32", 128, 1, 32, 5, 1, 1),
    (tuple((7 * i) % 11 for i in range(40)), tuple((13 * i) % 250 for i in range(40)), "bf16",
     128, 2, 16, 0, 40, 2),
]


@pytest.mark.parametrize("new,past,dtype,D,G,PS,shares,window,sinks", WINDOW)
def test_window(new, past, dtype, D, G, PS, shares, window, sinks):
    c = Masked(new, past, dtype, D, G, PS=PS, window=window, sinks=sinks)
    c.give_back()
    table = c.table
    c.table = torch.tensor(c.clean[2], device="cuda")
    spoil_the_rest(c)
    c.table = table
    out, lse = c.attend(num_shares=shares)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("window", [1, 63, 64, 127, 128, 129, 130, 192, 256, 257, 383, 500])
@pytest.mark.parametrize("shares", [0, 1, 5])
def test_window_whose_row_tiles_begin_apart(G, window, shares):
    """At D = 64 the second tile of rows may begin a key tile later than the first."""
    for new, past, sinks, PS in (((900, 333, 129), (0, 700, 64), 0, 16), ((1024,), (2000,), 0, 64),
                                 ((600, 200), (300, 1000), 5, 32)):
        test_window(new, past, "bf16", 64, G, PS, shares, window, sinks)


# batches of few rows (32 to a sequence on average, heads counted), whose items have 32 rows: some
# of the batch may have more, cut into several items
FEW = [
    # new, past, dtype, D, G, PS, shares
    ((1,), (0,), "bf16", 128, 1, 16, 0),
    ((1,), (5,), "bf16", 64, 8, 64, 0),
    ((4,), (3000,), "bf16", 128, 8, 16, 0),
    ((8,), (3001,), "bf16", 64, 4, 32, 0),
    ((32,), (700,), "bf16", 128, 1, 64, 5),
    ((32,), (700,), "bf16", 64, 1, 16, 0),
    ((16, 0, 3, 16, 9), (0, 40, 127, 128, 1000), "bf16", 128, 2, 16, 3),
    ((1, 1, 1, 1, 1, 1, 40), (0, 15, 16, 127, 128, 1400, 900), "bf16", 128, 4, 32, 0),
    ((1, 1, 1, 1, 1, 1, 40), (0, 15, 16, 127, 128, 1400, 900), "bf16", 64, 4, 16, 2),
    ((2, 2, 2, 2), (62, 190, 254, 4094), "bf16", 64, 8, 16, 40),
    (tuple(1 + i % 3 for i in range(40)), tuple((131 * i) % 1500 for i in range(40)), "bf16", 128,
     8, 16, 0),
    (tuple(1 + i % 3 for i in range(40)), tuple((131 * i) % 1500 for i in range(40)), "bf16", 64,
     2, 64, 0),
]


FEW += [
    # more sequences than one warp looks through for a block's place, most without rows
    (tuple(int(i % 7 == 3) for i in range(300)), tuple((37 * i) % 200 for i in range(300)), "bf16",
     128, 4, 16, 0),
    (tuple(int(i % 5 == 1) for i in range(1100)), tuple((11 * i) % 90 for i in range(1100)), "bf16",
     64, 2, 16, 0),
]
FEW += [(new, past, "fp32", D, G, PS, shares) for new, past, _, D, G, PS, shares in FEW]


@pytest.mark.parametrize("new,past,dtype,D,G,PS,shares", FEW)
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (1000, 300), (10 ** 6, 0)])
def test_window_of_few_rows(new, past, dtype, D, G, PS, shares, window, sinks):
    test_window(new, past, dtype, D, G, PS, shares, window, sinks)


@pytest.mark.parametrize("new,past,dtype,D,G,PS,shares", FEW)
def test_tree_of_few_rows(new, past, dtype, D, G, PS, shares):
    test_tree(new, past, dtype, D, G, PS, shares)


def test_few_rows_whose_maximum_keeps_growing():
    """Keys that grow along the sequence: the reference moves, and what was summed is rescaled."""
    for D, G, dtype in ((128, 4, "bf16"), (64, 8, "bf16"), (128, 2, "fp32")):
        for kind in ("window", "tree"):
            c = Masked((1, 4), (1500, 2000), dtype, D, G, window=1200 if kind == "window" else None,
                       sinks=3, parents=[[-1], bush(4, 2)] if kind == "tree" else None)
            grow = torch.linspace(0.1, 6.0, c.PS, device="cuda")
            for b, n in enumerate(c.lens):
                for p in range(-(-n // c.PS)):
                    c.k_pool[c.table[b, p].long()] *= (grow * (1 + p / 8))[None, :, None].to(
                        c.k_pool.dtype)
            c.clean = (f64(c.k_pool), f64(c.v_pool), c.clean[2])
            out, lse = c.attend()
            assert_no_device_error()
            c.check_attn(c.q, out, lse)


def test_window_of_single_tokens_without_offsets():
    """One row per sequence; the row of an empty sequence is zeros."""
    c = Masked((1, 1, 1, 1), (5000, 130, 77, 4096), G=8, window=300, sinks=4)
    c.give_back()
    out, lse = c.attend(cu_tokens=None)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    c.set_len([5001, 0, 78, 4097])
    again, lse2 = c.attend(cu_tokens=None)
    assert_no_device_error()
    assert (again[1] == 0).all() and torch.isinf(lse2[1]).all()
    keep = [0, 2, 3]
    same, lse3 = c.attend(cu_tokens=None)
    assert torch.equal(again[keep], same[keep]) and torch.equal(lse2[keep], lse3[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shares", [0, 1])
def test_a_window_that_reaches_the_start_is_causal(dtype, shares):
    c = Masked((300, 1, 77), (1000, 800, 0), dtype, window=4096)
    out, lse = c.attend(num_shares=shares)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    c.check_attn(c.q, ref, ref_lse)


def test_window_flags_pages_that_rows_see():
    """A page inside the window, or among the sinks, that is unmapped is flagged and not read."""
    for page in (0, 60):
        c = Masked((4,), (1000,), window=100, sinks=4)
        c.table[0, page] = -1
        c.attend()
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags == 1


def test_long_window_rows_leave_others_alone():
    """Rows behind the last sequence keep what they held."""
    c = Masked((33, 100), (900, 0), window=64, sinks=2, tail=5)
    out = torch.full((c.T + 5, c.Hq, c.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T + 5, c.Hq), 7.0, device="cuda")
    c.attend(out=out, lse=lse)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    assert (out[c.T:] == 7.0).all() and (lse[c.T:] == 7.0).all()


# ----------------------------------------------------------------------------- trees

def line(n):
    return list(range(-1, n - 1))


def bush(n, seed):
    rng = np.random.default_rng(seed)
    return [-1 if i == 0 or rng.random() < 0.15 else int(rng.integers(max(0, i - 9), i))
            for i in range(n)]


TREE = [
    # nodes, past, dtype, D, G, PS, shares
    ((1,), (0,), "bf16", 128, 4, 16, 0),
    ((8,), (2000,), "bf16", 128, 4, 16, 0),
    ((31,), (97,), "bf16", 128, 1, 16, 1),
    ((65,), (0,), "bf16", 64, 8, 64, 0),
    ((26, 0, 1, 64, 33), (500, 40, 63, 1, 900), "bf16", 128, 8, 64, 0),
    ((26, 0, 1, 64, 33), (500, 40, 63, 1, 900), "bf16", 64, 2, 32, 5),
    ((260, 129), (1000, 31), "bf16", 128, 4, 16, 0),
    ((260, 129), (1000, 31), "bf16", 128, 1, 16, 1),
    ((700,), (333,), "bf16", 64, 4, 16, 0),
    ((7, 31, 12, 1), (1000, 400, 63, 250), "fp32", 64, 4, 16, 0),
    ((140, 33), (77, 300), "fp32", 128, 8, 64, 3),
    ((140, 33), (77, 300), "fp32", 128, 1, 16, 1),
]


@pytest.mark.parametrize("new,past,dtype,D,G,PS,shares", TREE)
def test_tree(new, past, dtype, D, G, PS, shares):
    c = Masked(new, past, dtype, D, G, PS=PS, parents=[bush(n, 7 + n) for n in new])
    spoil_the_rest(c)
    out, lse = c.attend(num_shares=shares)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


@pytest.mark.parametrize("dtype,G", [("bf16", 4), ("bf16", 1), ("fp32", 2)])
@pytest.mark.parametrize("past", [0, 5, 2000])
def test_a_tree_that_is_one_line_is_causal(dtype, G, past):
    c = Masked((1024, 33), (past, 64), dtype, G=G, parents=[line(1024), line(33)])
    out, lse = c.attend()
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    assert_no_device_error()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_tree_of_roots_only(dtype):
    """Every node continues the cache: with nothing cached a row sees itself alone."""
    c = Masked((200, 40), (0, 300), dtype, parents=[[-1] * 200, [-1] * 40])
    out, lse = c.attend()
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    own = c.v_pool[c.table[0].long()].transpose(1, 2).reshape(-1, c.Hkv, c.D)[:200]
    if dtype == "bf16":
        assert torch.equal(out[:200], own.repeat_interleave(c.G, dim=1))


def test_single_rows_are_trees_without_offsets():
    c = Masked((1, 1, 1), (100, 0, 2050), G=2, parents=[[-1]] * 3)
    out, lse = c.attend(cu_tokens=None)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parents_that_are_not_earlier_rows_are_flagged(dtype):
    for bad in (5, 6, 100, -2, 2 ** 31 - 1, -2 ** 31):
        c = Masked((9, 4), (50, 3), dtype, parents=[bush(9, 1), line(4)])
        c.up[5] = bad
        out, lse = c.attend()
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags == 4
        c.parents[0][5] = -1                       # what it is taken as
        c.check_attn(c.q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_tree_of_too_many_nodes_is_left_out(dtype):
    c = Masked((3, 1025, 20), (50, 0, 7), dtype, parents=[line(3), line(1025), bush(20, 3)], Hkv=1)
    out = torch.full((c.T, c.Hq, c.D), 7.0, dtype=c.q.dtype, device="cuda")
    c.attend(out=out)
    st, flags = skv.kv_check_device_errors()
    assert st == -5 and flags == 2
    assert (out[3:1028] == 7.0).all()
    ref, lse, tol, _ = c.attn_bounds(c.q)
    rows = list(range(3)) + list(range(1028, 1048))
    assert (np.abs(f64(out) - ref) <= tol)[rows].all()


def test_strided_queries_streams_and_the_same_bits():
    """A fused projection's rows, another stream, and the same call many times over."""
    c = Masked((40, 64, 1, 100), (3000, 100, 77, 0), parents=[bush(n, n) for n in (40, 64, 1, 100)])
    first, lse = c.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        out, lse2 = c.attend(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, first) and torch.equal(lse, lse2)
    assert_no_device_error()
    assert not c.q.is_contiguous()
    packed, _ = skv.kv_tree_attn(c.kv, c.q.contiguous(), c.scale, c.up, cu_tokens=c.cu)
    assert torch.equal(packed, first)


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_captured_calls_follow_lengths_and_parents(kind):
    c = Masked((20, 30, 8), (600, 100, 1500), window=100 if kind == "window" else None, sinks=4,
               parents=[bush(20, 1), bush(30, 2), bush(8, 3)] if kind == "tree" else None)
    ws = torch.empty((skv.kv_prefill_attn_workspace_size(c.kv, c.Hq, c.T),), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((c.T, c.Hq, c.D), dtype=c.q.dtype, device="cuda")
    lse = torch.empty((c.T, c.Hq), device="cuda")
    c.attend(workspace=ws, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(workspace=ws, out=out, lse=lse)
    if kind == "tree":
        c.parents = [line(20), bush(30, 9), [-1] * 8]
        c.up.copy_(torch.tensor([p for t in c.parents for p in t], dtype=torch.int32))
    c.lens = [500, 131, 1400]
    c.set_len(c.lens)
    c.past = [480, 101, 1392]
    out.fill_(9.0)
    graph.replay()
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


def test_windows_and_trees_past_2_31_pool_rows_are_refused():
    c = Masked((2,), (3,), window=4)
    d = c.kv.desc
    d.num_phys_pages = 2 ** 31 // (c.Hkv * c.PS)
    with pytest.raises(binding.KVError):
        c.attend()
