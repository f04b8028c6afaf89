"""Packed append with rotation, and causal attention of packed rows, against the float64 oracle.

Error bounds, from the arithmetic of the operators:

* rotation in float32: the angle is off by 2^-25 (its conversion to half turns, times pi) and
  sine and cosine by two units, together under 2^-22; two products and a sum add 3 * 2^-24. All
  of it scales with |a| + |b| of the pair, so 2^-21 (|a| + |b|) holds them, and the rounding to
  the storage type adds half a step, finfo.eps / 2, relative to the value;
* attention: a logit is off by D roundings of sums no larger than sum |q k|, at most 2^-23 each
  (the tensor core's adder may truncate), D * 2^-23 * logit; a probability is off, relative to
  itself, by twice that (its own and the sum's), by the exponential (2^-21) and, for bf16, by its
  rounding (2^-8); sums over L keys add L * 2^-23. All of it scales with sum p |v|. The output's
  rounding adds eps / 2 of the value.
"""

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import prompt
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, f64, need_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


class Case:
    """A cache whose new tokens are mapped but not yet written, and their packed rows."""

    def __init__(self, new, past, dtype="bf16", D=128, G=4, Hkv=2, PS=16, seed=1, fused=True,
                 extra=3, tail=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.past, self.dtype, self.D, self.G, self.PS = new, past, dtype, D, G, PS
        self.Hkv, self.Hq, B = Hkv, Hkv * G, len(new)
        self.lens = [n + p for n, p in zip(new, past)]
        pages = [-(-n // PS) for n in self.lens]
        NP, T = sum(pages) + extra, sum(new)
        self.T, self.scale = T, D ** -0.5

        def rand(*shape):
            return torch.randn(shape, generator=gen, device="cuda").to(DT[dtype])

        self.k_pool, self.v_pool = rand(NP, Hkv, PS, D), rand(NP, Hkv, PS, D)
        order = torch.randperm(NP, generator=gen, device="cuda").to(torch.int32)
        self.table = torch.full((B, max(max(pages), 1)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cu_h = np.concatenate([[0], np.cumsum(new)])
        self.cu = torch.tensor(self.cu_h, dtype=torch.int32, device="cuda")
        # `tail` packed rows behind the last sequence's belong to nobody
        if fused:
            x = rand(T + tail, self.Hq + 2 * Hkv, D)
            self.q, self.k, self.v = x.split((self.Hq, Hkv, Hkv), dim=1)
        else:
            self.q, self.k, self.v = (rand(T + tail, h, D) for h in (self.Hq, Hkv, Hkv))
        self.kv = skv.PagedKV(self.k_pool, self.v_pool, self.table, self.seq_lens)

    def slots(self):
        """Index arrays of the new tokens' places in a pool (page, slot), token by token."""
        seq, pos = prompt.row_places(self.cu_h, self.lens)
        table = self.table.cpu().numpy()
        return seq, pos, table[seq, pos // self.PS], pos % self.PS

    def set_len(self, lens):
        self.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))

    def past_stats(self):
        """Statistics as the past left them, by the library's own full build."""
        self.set_len(self.past)
        stats = skv.kv_build_page_stats(self.kv, stats=torch.full(
            (self.k_pool.shape[0], self.Hkv, 2, self.D), 77.0, dtype=DT[self.dtype],
            device="cuda"))
        self.set_len(self.lens)
        return stats

    def attn_bounds(self, q):
        out, lse, mass, logit = prompt.prefill(f64(q), f64(self.k_pool), f64(self.v_pool),
                                               self.table.cpu().numpy(), self.lens, self.cu_h,
                                               self.PS, self.scale)
        L = max(self.lens)
        dx = self.D * 2.0 ** -23 * logit
        rel = 2 * dx + 2.0 ** -21 + L * 2.0 ** -23
        p = half_step("bf16") if self.dtype == "bf16" else 0.0
        tol = (rel + p)[..., None] * mass * 1.01 + half_step(self.dtype) * np.abs(out) * 1.01
        return out, lse, tol + 1e-30, rel + 2.0 ** -23 * np.abs(lse)

    def check_attn(self, q, out, lse):
        ref, ref_lse, tol, tol_lse = self.attn_bounds(q)
        T = ref.shape[0]
        err, err_lse = np.abs(f64(out)[:T] - ref), np.abs(f64(lse)[:T] - ref_lse)
        assert (err <= tol)[~np.isnan(ref)].all(), np.nanmax(err / tol)
        assert (err_lse <= tol_lse)[~np.isnan(ref_lse)].all(), np.nanmax(err_lse / tol_lse)
        assert not np.isnan(f64(out)[:T][~np.isnan(ref)]).any()


def freqs(rot):
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


# --------------------------------------------------------------------------- append

APPEND = [
    # new, past, dtype, D, G, PS, rot, interleaved
    ((16,), (0,), "bf16", 128, 4, 16, 128, False),
    ((1, 1, 1), (0, 15, 16), "bf16", 128, 4, 16, 128, False),
    ((5, 0, 100, 1, 33), (3, 7, 0, 63, 31), "bf16", 128, 1, 32, 128, True),
    ((129, 64, 63), (1, 64, 200), "bf16", 64, 8, 64, 64, False),
    ((40, 17), (0, 9), "bf16", 64, 2, 16, 32, True),
    ((40, 17), (0, 9), "bf16", 128, 2, 16, 32, False),
    ((7, 50), (100, 0), "fp32", 64, 2, 16, 64, False),
    ((7, 50), (100, 0), "fp32", 128, 4, 32, 96, True),
    ((7, 50), (100, 0), "fp32", 128, 8, 64, 0, False),
    (tuple(i % 5 for i in range(45)), tuple(3 * i for i in range(45)), "bf16", 64, 1, 16, 64,
     False),
]


def check_append(c, q_out, stats, before, rot, inter, pos_of_row=None, tokens=None):
    """Everything the append wrote, and that it wrote nothing else. `tokens`: the rows that
    are expected to have been appended (all by default)."""
    seq, pos, phys, slot = c.slots()
    rows = np.arange(c.T) if tokens is None else np.asarray(tokens)
    angle_pos = pos if pos_of_row is None else pos_of_row
    k0, v0, q0 = before
    for name, x, got in (("q", c.q_in, q_out[:c.T]),
                         ("k", c.k, c.k_pool[phys, :, slot])):
        ref, mag = prompt.rope(f64(x)[:c.T], angle_pos, freqs(rot) if rot else [], inter)
        # far angles: the frequency's division by 2 pi and the oracle's own product round
        # three times at 2^-53 of up to pos radians
        e = (2.0 ** -21 + 3 * 2.0 ** -53 * np.abs(angle_pos))[:, None, None] * mag
        tol = e * (np.abs(ref - f64(x)[:c.T]) > 0) + half_step(c.dtype) * (np.abs(ref) + e)
        err = np.abs(f64(got) - ref)
        assert (err[rows] <= tol[rows]).all(), (name, (err[rows] - tol[rows]).max())
    assert torch.equal(c.v_pool[phys, :, slot][rows], c.v[:c.T][rows])
    # slots that hold no new token, and packed rows of nobody, are as they were
    for pool, old in ((c.k_pool, k0), (c.v_pool, v0)):
        mask = torch.ones(pool.shape[0], c.PS, dtype=torch.bool, device="cuda")
        mask[phys[rows], slot[rows]] = False
        assert torch.equal(pool.transpose(1, 2)[mask], old.transpose(1, 2)[mask])
    if q0 is not None:
        rest = np.setdiff1d(np.arange(q_out.shape[0]), rows)
        assert torch.equal(q_out[rest], q0[rest])


def pages_of(c, lens):
    table = c.table.cpu().numpy()
    return np.unique(np.concatenate([table[b, : -(-n // c.PS)] for b, n in enumerate(lens)]))


@pytest.mark.parametrize("new,past,dtype,D,G,PS,rot,inter", APPEND)
def test_append_rope_matches_the_oracle(new, past, dtype, D, G, PS, rot, inter):
    c = Case(new, past, dtype, D, G, PS=PS, tail=2)
    stats = c.past_stats()
    untouched = torch.full_like(c.q, -9.0).contiguous()
    q_out = untouched.clone()
    before = (c.k_pool.clone(), c.v_pool.clone(), untouched)
    old = stats.clone()
    c.q_in = c.q.clone()
    turns = skv.kv_rope_turns(freqs(rot), device="cuda") if rot else None
    got = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu,
                             interleaved=inter, q_out=q_out)
    assert got is q_out
    assert_no_device_error()
    check_append(c, q_out, stats, before, rot, inter)
    mapped = pages_of(c, c.lens)
    rebuilt = skv.kv_build_page_stats(c.kv)
    np.testing.assert_array_equal(f64(stats)[mapped], f64(rebuilt)[mapped])
    rest = np.setdiff1d(np.arange(stats.shape[0]), mapped)
    assert torch.equal(stats[rest], old[rest])


@pytest.mark.parametrize("dtype,D,G,PS,inter", [("bf16", 128, 4, 16, False),
                                                ("bf16", 64, 8, 64, True),
                                                ("fp32", 128, 1, 32, False),
                                                ("fp32", 64, 2, 16, True)])
def test_append_one_token_per_sequence(dtype, D, G, PS, inter):
    past = (0, 15, 16, 31, 100, 63, 64)
    c = Case((1,) * len(past), past, dtype, D, G, PS=PS)
    stats = c.past_stats()
    ref_stats, k1, v1 = stats.clone(), c.k_pool.clone(), c.v_pool.clone()
    before = (k1.clone(), v1.clone(), None)
    c.q_in = c.q.clone()
    turns = skv.kv_rope_turns(freqs(D), device="cuda")
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, interleaved=inter)
    assert_no_device_error()
    check_append(c, q, stats, before, D, inter)
    # the packed form of the same call writes the same bits
    kv = skv.PagedKV(k1, v1, c.table, c.seq_lens)
    q2 = skv.kv_append_rope(kv, c.q, c.k, c.v, ref_stats, turns, cu_tokens=c.cu,
                            interleaved=inter)
    for a, b in ((q, q2), (c.k_pool, k1), (c.v_pool, v1), (stats, ref_stats)):
        assert torch.equal(a, b)
    rebuilt = skv.kv_build_page_stats(c.kv)
    mapped = pages_of(c, c.lens)
    np.testing.assert_array_equal(f64(stats)[mapped], f64(rebuilt)[mapped])


def test_append_without_rotation_equals_append_token():
    c = Case((1, 1, 1), (5, 16, 47), "bf16", 128, 4)
    stats = c.past_stats()
    k1, v1, s1 = c.k_pool.clone(), c.v_pool.clone(), stats.clone()
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats)
    assert torch.equal(q, c.q)
    skv.kv_append_token(skv.PagedKV(k1, v1, c.table, c.seq_lens), c.k.contiguous(),
                        c.v.contiguous(), s1)
    for a, b in ((c.k_pool, k1), (c.v_pool, v1), (stats, s1)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("packed", [True, False])
def test_append_leaves_empty_sequences_alone(packed):
    c = Case((1, 0, 1) if packed else (1, 1, 1), (4, 0, 20) if packed else (4, 0, 20))
    if not packed:
        c.set_len((5, 0, 21))              # the middle sequence has no token
    stats = c.past_stats()
    if not packed:
        c.set_len((5, 0, 21))
    q_out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    k0 = c.k_pool.clone()
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, cu_tokens=c.cu if packed else None,
                       q_out=q_out)
    assert_no_device_error()
    if packed:
        assert torch.equal(q_out, c.q)
    else:
        assert torch.equal(q_out[[0, 2]], c.q[[0, 2]]) and (q_out[1] == -9.0).all()
        P = int(c.table[1, 0])
        assert torch.equal(c.k_pool[P], k0[P])


def test_append_far_and_given_positions_in_place():
    """Positions near 2^31, negative ones and repeated ones; q rotated in place."""
    c = Case((6,), (0,), "fp32", 64, 2)
    pos = [2 ** 31 - 1, 10 ** 6, 10 ** 6, 0, -5, 123456789]
    stats = c.past_stats()
    before = (c.k_pool.clone(), c.v_pool.clone(), None)
    c.q_in = c.q.clone()
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, skv.kv_rope_turns(freqs(64), device="cuda"),
                       cu_tokens=c.cu, q_out=c.q,
                       positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert_no_device_error()
    check_append(c, c.q, stats, before, 64, False, pos_of_row=np.array(pos))


def test_append_flags_bad_data_and_writes_nothing_there():
    c = Case((20, 20, 20), (0, 0, 0))
    stats = c.past_stats()
    k0, s0 = c.k_pool.clone(), stats.clone()
    for cu in ([0, 20, 10, 60], [0, 20, 61, 60], [0, -1, 40, 60], [5, 20, 40, 60]):
        skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats,
                           cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags & 2, cu
    # a sequence shorter than its new tokens is left out, the others are appended
    c.k_pool.copy_(k0)
    stats.copy_(s0)
    c.set_len((20, 19, 20))
    q_out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, cu_tokens=c.cu, q_out=q_out)
    st, flags = skv.kv_check_device_errors()
    assert st == -5 and flags == 2
    mid = c.table[1, :2].long()
    assert torch.equal(c.k_pool[mid], k0[mid]) and (q_out[20:40] == -9.0).all()
    assert torch.equal(q_out[40:], c.q[40:])
    # an unmapped page: its tokens are skipped, the rest of the sequence is written
    c.k_pool.copy_(k0)
    c.set_len((20, 20, 20))
    gone = int(c.table[2, 0])
    c.table[2, 0] = 10 ** 6
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, cu_tokens=c.cu, q_out=q_out)
    st, flags = skv.kv_check_device_errors()
    assert st == -5 and flags == 1
    assert torch.equal(c.k_pool[gone], k0[gone])
    assert torch.equal(c.k_pool[int(c.table[2, 1]), :, :4].transpose(0, 1), c.k[56:60])
    assert torch.equal(q_out, c.q)
    c.table[2, 0] = -1
    skv.kv_append_rope(c.kv, c.q[:3], c.k[:3], c.v[:3], stats)     # page 1 of each: mapped
    assert_no_device_error()


@pytest.mark.parametrize("dtype,D,G,PS,inter", [("bf16", 128, 4, 16, False),
                                                ("bf16", 128, 1, 64, True),
                                                ("bf16", 64, 8, 32, False),
                                                ("fp32", 128, 2, 64, False),
                                                ("fp32", 64, 1, 16, True)])
def test_append_many_rows(dtype, D, G, PS, inter):
    """From 8192 (token, KV head) pairs on, a warp takes several steps of its page."""
    c = Case((2501, 0, 1, 1595), (37, 5, 63, 0), dtype, D, G, PS=PS)
    c.q_in = c.q
    stats = c.past_stats()
    before = (c.k_pool.clone(), c.v_pool.clone(), None)
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, skv.kv_rope_turns(freqs(D), device="cuda"),
                           cu_tokens=c.cu, interleaved=inter)
    assert_no_device_error()
    check_append(c, q, stats, before, D, inter)
    used = pages_of(c, c.lens)
    assert torch.equal(stats[used], skv.kv_build_page_stats(c.kv)[used])


def test_append_to_many_sequences():
    """More sequences than one round of the search's loads, many without new tokens."""
    c = Case(tuple(i * i % 4 for i in range(2500)), tuple(7 * i % 40 for i in range(2500)),
             D=64, G=1)
    c.q_in = c.q
    stats = c.past_stats()
    before = (c.k_pool.clone(), c.v_pool.clone(), None)
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, skv.kv_rope_turns(freqs(64), device="cuda"),
                           cu_tokens=c.cu)
    assert_no_device_error()
    check_append(c, q, stats, before, 64, False)
    used = pages_of(c, c.lens)
    assert torch.equal(stats[used], skv.kv_build_page_stats(c.kv)[used])


def test_append_past_32_bit_offsets():
    """Slots and statistics of the last pages of pools of more than 2^31 elements."""
    NP = 2 ** 31 // (2 * 16 * 128) + 40
    c = Case((20, 1), (5, 16), extra=0)
    need = c.k_pool.shape[0]
    small_k, small_v, table = c.k_pool, c.v_pool, c.table.clone()
    c.k_pool = torch.empty((NP, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    c.v_pool = torch.empty_like(c.k_pool)
    c.k_pool[-need:], c.v_pool[-need:] = small_k, small_v
    c.table = torch.where(table >= 0, table + (NP - need), table).to(torch.int32)
    c.kv = skv.PagedKV(c.k_pool, c.v_pool, c.table, c.seq_lens)
    turns = skv.kv_rope_turns(freqs(128), device="cuda")
    stats = torch.empty((NP, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu)
    assert_no_device_error()
    c.k_pool, c.v_pool, c.table = small_k.clone(), small_v.clone(), table
    big = c.kv
    c.kv = skv.PagedKV(c.k_pool, c.v_pool, table, c.seq_lens)
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, c.past_stats(), turns, cu_tokens=c.cu)
    assert_no_device_error()
    assert torch.equal(big.k_pool[-need:], c.k_pool)
    assert torch.equal(big.v_pool[-need:], c.v_pool)


@pytest.mark.parametrize("cu", [(48, 54, 60, 60, 60, 60), (60, 60, 60, 60, 60, 60),
                                (0, 20, 40, 60, 10, 12), (0, 50, 55, 60, 0, 4)])
def test_append_with_offsets_that_number_no_page(cu):
    """Offsets that start above zero or fall leave numbers of the grid before the first page of
    the sequence they are found in: no table entry, slot or statistic belongs to them."""
    c = Case((12, 12, 12, 12, 12), (40, 0, 3, 20, 16))
    stats = c.past_stats()
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats,
                       cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    st, flags = skv.kv_check_device_errors()
    assert st == -5 and flags == 2
    # what was written is the statistics of what is cached, as far as each page is filled
    cached = skv.kv_build_page_stats(c.kv, stats=stats.clone())
    for b, (n, r) in enumerate(zip(np.diff(cu), cu)):
        if n < 0 or n > c.lens[b]:
            continue
        for page in range((c.lens[b] - n) // c.PS, -(-c.lens[b] // c.PS) if n else 0):
            P = int(c.table[b, page])
            if page * c.PS >= c.lens[b] - n:
                assert torch.equal(stats[P], cached[P]), (b, page)


# ------------------------------------------------------------------------ attention

ATTN = [
    # new, past, dtype, D, G, PS, blocks the work is shared among (0: as many as the GPU holds)
    ((1,), (0,), "bf16", 128, 4, 16, 0),
    ((128,), (0,), "bf16", 128, 1, 16, 1),
    ((257,), (0,), "bf16", 128, 4, 16, 0),
    ((257,), (0,), "bf16", 64, 1, 32, 1),
    ((300, 1, 0, 129, 64), (0, 500, 40, 127, 128), "bf16", 128, 4, 16, 1),
    ((300, 1, 0, 129, 64), (0, 500, 40, 127, 128), "bf16", 128, 4, 16, 0),
    ((300, 1, 0, 129, 64), (0, 500, 40, 127, 128), "bf16", 64, 8, 64, 3),
    ((40, 700), (1000, 3), "bf16", 128, 8, 32, 2),
    ((40, 700), (1000, 3), "bf16", 128, 1, 64, 29),
    ((500, 33), (0, 17), "bf16", 64, 2, 32, 0),
    ((1, 1, 1, 1), (0, 127, 128, 900), "bf16", 128, 8, 16, 4),
    ((5, 5, 5), (63, 1500, 700), "bf16", 64, 1, 16, 7),
    ((5, 33, 64), (3063, 1500, 1700), "bf16", 128, 4, 16, 100),
    ((1,), (2047,), "bf16", 128, 2, 16, 64),
    ((1,), (4090,), "bf16", 128, 8, 64, 0),
    ((65, 1, 200), (0, 300, 64), "fp32", 64, 4, 16, 1),
    ((65, 1, 200), (0, 300, 64), "fp32", 128, 8, 64, 3),
    ((65, 1, 200), (0, 300, 64), "fp32", 128, 8, 64, 0),
    ((1, 1, 1), (0, 700, 15), "fp32", 128, 1, 32, 5),
    ((1,), (2500,), "fp32", 64, 2, 16, 0),
    (tuple((7 * i) % 11 for i in range(40)), tuple((13 * i) % 50 for i in range(40)), "bf16",
     128, 2, 16, 1),
    (tuple((7 * i) % 11 for i in range(40)), tuple((13 * i) % 50 for i in range(40)), "bf16",
     128, 2, 16, 0),
]


def spoil_the_rest(c):
    """NaN and infinities in every slot that holds no token, as fresh memory may hold them."""
    used = torch.zeros(c.k_pool.shape[0], c.PS, dtype=torch.bool, device="cuda")
    table = c.table.cpu().numpy()
    for b, n in enumerate(c.lens):
        for p in range(-(-n // c.PS)):
            used[table[b, p], : min(c.PS, n - p * c.PS)] = True
    for pool, bad in ((c.k_pool, float("nan")), (c.v_pool, float("inf"))):
        pool.transpose(1, 2)[~used] = bad


@pytest.mark.parametrize("new,past,dtype,D,G,PS,shares", ATTN)
def test_prefill_attn_matches_the_oracle(new, past, dtype, D, G, PS, shares):
    c = Case(new, past, dtype, D, G, PS=PS, tail=3)
    c.q.mul_(2.0)
    ref_case = c.attn_bounds(c.q)          # before the unused slots are spoiled
    spoil_the_rest(c)
    out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], -9.0, device="cuda")
    skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares, out=out, lse=lse)
    assert_no_device_error()
    ref, ref_lse, tol, tol_lse = ref_case
    err, err_lse = np.abs(f64(out)[:c.T] - ref[:c.T]), np.abs(f64(lse)[:c.T] - ref_lse[:c.T])
    assert (err <= tol[:c.T]).all(), np.nanmax(err / tol[:c.T])
    assert (err_lse <= tol_lse[:c.T]).all(), np.nanmax(err_lse / tol_lse[:c.T])
    assert (out[c.T:] == -9.0).all() and (lse[c.T:] == -9.0).all()      # rows of nobody


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shares", [0, 1, 5, 1000])
def test_prefill_attn_one_token_per_sequence(dtype, shares):
    c = Case((1,) * 6, (0, 1, 15, 300, 1200, 64), dtype, 128, 4, fused=False)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=shares)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)
    packed, lse2 = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares)
    assert torch.equal(out, packed) and torch.equal(lse, lse2)
    # and an empty sequence among them: zeros, lse -inf
    c.set_len((1, 0, 16, 301, 1201, 65))
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=shares)
    assert_no_device_error()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    # the other rows may be cut elsewhere now: equal to the oracle again, not bit for bit
    want, _, tol, _ = c.attn_bounds(c.q)
    assert (np.abs(f64(out) - want) <= tol)[2:].all()
    assert torch.equal(out[2:], packed[2:]) or shares != 1


@pytest.mark.parametrize("dtype,rows", [("bf16", 300), ("bf16", 20), ("fp32", 70)])
def test_prefill_attn_rising_and_extreme_scores(dtype, rows):
    """Keys that grow along the sequence, so that the running maximum rises in every tile, and
    ones so large that all but one probability vanish."""
    for size in (0.05, 3.0):
        c = Case((rows,), (900,), dtype, 128, 4)
        t = torch.arange(c.lens[0], device="cuda")
        unit = c.q[:, :1].float().mean(0).sign()                       # [1][D]
        for g in range(c.Hkv):
            c.k_pool[c.table[0, t // 16].long(), g, t % 16] = \
                (unit * (size * t[:, None] / 100)).to(c.k_pool.dtype)
        c.q.copy_(unit.expand_as(c.q) * 0.5)
        out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
        assert_no_device_error()
        c.check_attn(c.q, out, lse)


def test_prefill_attn_many_sequences():
    n = 1100                                  # more than two rounds of the offsets' search
    c = Case(tuple(1 + i % 3 for i in range(n)), tuple(i % 40 for i in range(n)), "bf16", 64, 2)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_attn_past_32_bit_offsets(dtype):
    """Pages whose elements lie beyond 2^32 bytes, and beyond 2^31 elements, of the pool."""
    D, Hkv, PS = 128, 8, 64
    NP = (2 ** 31) // (Hkv * PS * D) + 40
    c = Case((70,), (200,), dtype, D, 2, Hkv=Hkv, PS=PS)
    k = torch.zeros((NP, Hkv, PS, D), dtype=DT[dtype], device="cuda")
    v = torch.zeros_like(k)
    far = torch.arange(NP - c.k_pool.shape[0], NP, device="cuda")
    k[far], v[far] = c.k_pool, c.v_pool
    table = torch.where(c.table >= 0, c.table + int(far[0]), c.table)
    kv = skv.PagedKV(k, v, table, c.seq_lens)
    stats = torch.zeros((NP, Hkv, 2, D), dtype=DT[dtype], device="cuda")
    q = skv.kv_append_rope(kv, c.q, c.k, c.v, stats, cu_tokens=c.cu)
    out, lse = skv.kv_prefill_attn(kv, q, c.scale, cu_tokens=c.cu)
    assert_no_device_error()
    c.k_pool.copy_(k[far])
    c.v_pool.copy_(v[far])
    seq, pos, phys, slot = c.slots()
    assert torch.equal(c.k_pool[phys, :, slot], c.k)
    c.check_attn(q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shares", [0, 1, 3])
def test_prefill_attn_of_a_batch_without_new_tokens(dtype, shares):
    """A padded batch between two requests: rows there are, but no sequence owns one."""
    c = Case((0, 0, 0), (0, 40, 500), dtype, tail=300)
    out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], -9.0, device="cuda")
    for _ in range(3):
        skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares, out=out,
                            lse=lse)
    assert_no_device_error()
    assert (out == -9.0).all() and (lse == -9.0).all()


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("bf16", 64, 1), ("fp32", 64, 2)])
def test_prefill_attn_of_sequences_that_share_pages(dtype, D, G):
    """A common prefix mapped by several sequences, and a page mapped twice by one."""
    c = Case((40, 3, 1, 200), (160, 317, 319, 120), dtype, D, G)
    c.table[1:, :6] = c.table[0, :6]
    c.table[3, 7] = c.table[3, 2]
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    assert_no_device_error()
    c.check_attn(c.q, out, lse)


def test_prefill_attn_flags_bad_data():
    c = Case((20, 20, 20), (0, 0, 0))
    for cu in ([0, 20, 10, 60], [0, 20, 61, 60], [0, -1, 40, 60], [5, 20, 40, 60]):
        for shares in (1, 2):
            skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=shares,
                                cu_tokens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
            st, flags = skv.kv_check_device_errors()
            assert st == -5 and flags & 2, cu
    ref, _ = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    want, _, tol, _ = c.attn_bounds(c.q)
    c.set_len((20, 19, 20))
    for shares in (1, 2):
        out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
        skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, out=out, num_shares=shares)
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags == 2
        assert (out[20:40] == -9.0).all()
        for rows in (slice(0, 20), slice(40, 60)):
            assert (np.abs(f64(out[rows]) - want[rows]) <= tol[rows]).all()
    c.set_len((20, 20, 20))
    for bad in (-1, 10 ** 6):
        c.table[1, 1] = bad
        out, _ = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
        st, flags = skv.kv_check_device_errors()
        assert st == -5 and flags == 1
        assert torch.equal(out[:20], ref[:20]) and torch.equal(out[40:], ref[40:])


# ------------------------------------------------------------- together, streams, graphs

def serve(c, chunks, turns, shares=0):
    """A prompt of one sequence in chunks: append, then attend, chunk by chunk."""
    stats = torch.zeros((c.k_pool.shape[0], c.Hkv, 2, c.D), dtype=DT[c.dtype], device="cuda")
    outs, qs, at = [], [], 0
    for n in chunks:
        c.set_len((at + n,))
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        rows = slice(at, at + n)
        q = skv.kv_append_rope(c.kv, c.q[rows], c.k[rows], c.v[rows], stats, turns,
                               cu_tokens=cu)
        outs.append(skv.kv_prefill_attn(c.kv, q, c.scale, cu_tokens=cu, num_shares=shares))
        qs.append(q)
        at += n
    return torch.cat(qs), torch.cat([o for o, _ in outs]), torch.cat([x for _, x in outs]), stats


@pytest.mark.parametrize("dtype,D,G,PS", [("bf16", 128, 4, 16), ("bf16", 64, 8, 64),
                                          ("fp32", 128, 2, 32)])
def test_a_prompt_in_chunks_then_decoded(dtype, D, G, PS):
    """Append and attention chunk by chunk equal one pass over the prompt; the decode step on
    the cache and statistics they leave equals the attention of the same single token."""
    c = Case((333,), (0,), dtype, D, G, PS=PS)
    turns = skv.kv_rope_turns(freqs(D), device="cuda")
    q, whole, whole_lse, stats = serve(c, (333,), turns)
    k1, s1 = c.k_pool.clone(), stats.clone()
    q2, out, lse, stats = serve(c, (1, 15, 17, 100, 1, 199), turns)
    assert_no_device_error()
    assert torch.equal(c.k_pool, k1)
    mapped = pages_of(c, (333,))
    assert torch.equal(stats[mapped], s1[mapped])
    assert torch.equal(q, q2)
    c.set_len((333,))
    _, _, tol, tol_lse = c.attn_bounds(q)
    c.check_attn(q, whole, whole_lse)
    c.check_attn(q, out, lse)
    # decode: one more token through the single-token forms
    last = skv.kv_append_rope(c.kv, c.q[332:], c.k[332:], c.v[332:], stats, turns)
    single, s_lse = skv.kv_prefill_attn(c.kv, last, c.scale)
    dense, d_lse = skv.kv_decode_step(c.kv, last, c.scale, keep_ratio=1.0)
    kept, _ = skv.kv_decode_step(c.kv, last, c.scale, stats, budget_pages=c.table.shape[1])
    assert_no_device_error()
    both = tol[332:] * 2
    assert (np.abs(f64(single) - f64(dense)) <= both).all()
    assert (np.abs(f64(kept) - f64(dense)) <= both).all()
    assert np.abs(f64(s_lse) - f64(d_lse)).max() <= 2 * tol_lse[332:].max()


@pytest.mark.parametrize("shares", [0, 1, 4])
def test_same_results_every_time_and_on_other_streams(shares):
    c = Case((200, 31), (100, 900), "bf16", 128, 4)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams * 3:                       # two calls at once, each with its workspace
        with torch.cuda.stream(s):
            got.append(skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu,
                                           num_shares=shares))
    torch.cuda.synchronize()
    assert_no_device_error()
    for o, x in got:
        assert torch.equal(o, out) and torch.equal(x, lse)


@pytest.mark.parametrize("new,past,PS", [((1,), (20000,), 16), ((5, 2, 1, 7), (9000, 3000, 12345, 1),
                                                               16),
                                         ((700, 1, 64, 300), (0, 5000, 900, 33), 64)])
def test_the_same_bits_call_after_call(new, past, PS):
    """Calls that follow one another without a pause: a tile read before it has landed, or a
    buffer given back too early, shows as other bits in one of many calls."""
    c = Case(new, past, "bf16", 128, 4, Hkv=8, PS=PS)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    ws = torch.empty((skv.kv_prefill_attn_workspace_size(c.kv, c.Hq, c.T),), dtype=torch.uint8,
                     device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        for _ in range(5):
            out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, workspace=ws)
        differ += (out != ref).sum() + (lse != ref_lse).sum()
    assert_no_device_error()
    assert int(differ) == 0


def test_captured_and_replayed_with_new_contents():
    """Append and attention captured into one graph; a replay reads the buffers as they are
    then (other rows, a longer cache), and two graphs share a workspace one after the other."""
    c = Case((1, 1, 1), (40, 500, 90), "bf16", 128, 4, extra=8)
    turns = skv.kv_rope_turns(freqs(128), device="cuda")
    stats = c.past_stats()
    ws = torch.empty((max(1, skv.kv_prefill_attn_workspace_size(c.kv, c.Hq, 3, 4)),),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        q = torch.empty(c.q.shape, dtype=c.q.dtype, device="cuda")
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")

        def step():
            skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, q_out=q)
            skv.kv_prefill_attn(c.kv, q, c.scale, num_shares=4, out=out, lse=lse, workspace=ws)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        outs.append((q, out, lse))
    for i, (g, (q, out, lse)) in enumerate(zip(graphs, outs)):
        c.q.copy_(torch.randn(c.q.shape, device="cuda"))
        c.k.copy_(torch.randn(c.k.shape, device="cuda"))
        lens = [41 + i, 501 + i, 91 + i]
        c.set_len(lens)
        g.replay()
        torch.cuda.synchronize()
        assert_no_device_error()
        c.lens = lens
        c.check_attn(q, out, lse)


def test_binding_refuses_what_it_cannot_pass_on():
    c = Case((4, 4), (0, 9))
    stats = c.past_stats()
    turns = skv.kv_rope_turns(freqs(128), device="cuda")
    bad = [
        dict(q=c.q[:, :, ::2]), dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q[:, 0]),
        dict(k=c.k[:3]), dict(v=c.v[:, :1]), dict(cu=c.cu[:2]), dict(cu=c.cu.long()),
        dict(cu=None), dict(stats=stats[1:]), dict(turns=turns.double()),
        dict(turns=turns.cpu()), dict(out=c.q[:4]), dict(pos=c.cu),
    ]
    for kw in bad:
        a = dict(q=c.q, k=c.k, v=c.v, cu=c.cu, stats=stats, turns=turns, out=None, pos=None)
        a.update(kw)
        with pytest.raises(ValueError):
            skv.kv_append_rope(c.kv, a["q"], a["k"], a["v"], a["stats"], a["turns"],
                               cu_tokens=a["cu"], q_out=a["out"], positions=a["pos"])
    for kw in (dict(q=c.q[:, :, ::2]), dict(cu=None), dict(out=c.q), dict(lse=c.cu)):
        a = dict(q=c.q, cu=c.cu, out=None, lse=None)
        a.update(kw)
        with pytest.raises(ValueError):
            skv.kv_prefill_attn(c.kv, a["q"], c.scale, cu_tokens=a["cu"], out=a["out"],
                                lse=a["lse"])
    small = torch.empty((256,), dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.KVError) as e:
        skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=3, workspace=small)
    assert e.value.status == -4
    # nothing to do: no rows at all
    none = c.q[:0]
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = skv.kv_prefill_attn(c.kv, none, c.scale, cu_tokens=zero)
    assert out.shape == (0, c.Hq, 128) and lse.shape == (0, c.Hq)
    assert skv.kv_append_rope(c.kv, none, c.k[:0], c.v[:0], stats, cu_tokens=zero).shape[0] == 0
    assert_no_device_error()
