"""The packed calls at their edges: waits that run out, tables and lengths at their limits,
streams given by argument, NaN, and the accuracy that the header states."""

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import prompt
from sparse_kv_cache_build_gb300 import binding

from gpu_helpers import assert_no_device_error, f64, need_gpu
from test_gpu_prompt import Case, check_append, freqs, pages_of

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


# ---------------------------------------------------------------- lengths out of range

@pytest.mark.parametrize("over", [1, 7, 2 ** 31 - 1, -1])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp32", 64)])
def test_append_leaves_out_a_sequence_longer_than_its_table(dtype, D, packed, over):
    """Its new tokens have no place: cached tokens, statistics and q_out stay as they were, and
    the other sequences are appended."""
    new = (3, 9, 1) if packed else (1, 1, 1)
    c = Case(new, (13, 23, 31), dtype, D, PS=16)       # two pages of 16 each: the second is full
    stats = c.past_stats()
    want_q = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    q_out = want_q.clone()
    k0, v0, s0 = c.k_pool.clone(), c.v_pool.clone(), stats.clone()
    lens = list(c.lens)
    turns = skv.kv_rope_turns([1.0] * (D // 2), device="cuda")
    cu = c.cu if packed else None
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=cu, q_out=want_q)
    assert_no_device_error()
    k1, v1, s1 = c.k_pool.clone(), c.v_pool.clone(), stats.clone()
    c.k_pool.copy_(k0)
    c.v_pool.copy_(v0)
    stats.copy_(s0)
    lens[1] = over if over in (-1, 2 ** 31 - 1) else 2 * 16 + over
    c.set_len(lens)
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=cu, q_out=q_out)
    assert skv.kv_check_device_errors() == (-5, 2)
    mid, rest = c.table[1, :2].long(), c.table[[0, 2]].flatten().long()
    rest = rest[rest >= 0]
    for got, old, full in ((c.k_pool, k0, k1), (c.v_pool, v0, v1), (stats, s0, s1)):
        assert torch.equal(got[mid], old[mid]) and torch.equal(got[rest], full[rest])
    rows = slice(int(c.cu_h[1]), int(c.cu_h[2]))
    assert (q_out[rows] == -9.0).all()
    for r in (slice(0, rows.start), slice(rows.stop, None)):
        assert torch.equal(q_out[r], want_q[r])


@pytest.mark.parametrize("over", [1, 7, 2 ** 31 - 1, -1])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("dtype,shares", [("bf16", 1), ("bf16", 3), ("fp32", 0)])
def test_attention_leaves_out_a_sequence_longer_than_its_table(dtype, shares, packed, over):
    c = Case((3, 9, 1) if packed else (1, 1, 1), (13, 23, 31), dtype, 128, PS=16)
    want, _, tol, _ = c.attn_bounds(c.q)
    lens = list(c.lens)
    lens[1] = over if over in (-1, 2 ** 31 - 1) else 2 * 16 + over
    c.set_len(lens)
    out = torch.full(c.q.shape, -9.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full(c.q.shape[:2], -9.0, device="cuda")
    skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu if packed else None,
                        num_shares=shares, out=out, lse=lse)
    assert skv.kv_check_device_errors() == (-5, 2)
    rows = slice(int(c.cu_h[1]), int(c.cu_h[2]))
    assert (out[rows] == -9.0).all() and (lse[rows] == -9.0).all()
    for r in (slice(0, rows.start), slice(rows.stop, None)):
        assert (np.abs(f64(out[r]) - want[r]) <= tol[r]).all()


# ------------------------------------------------------------------- arguments as users have them

def test_scalars_of_other_kinds():
    """numpy's numbers and one-element tensors, as the older calls take them."""
    c = Case((7, 1), (20, 40), "bf16", 128, 4)
    turns = skv.kv_rope_turns([0.5] * 64, device="cuda")
    stats = c.past_stats()
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu, interleaved=True)
    ref = skv.kv_prefill_attn(c.kv, q, 0.125, cu_tokens=c.cu, num_shares=3)
    for yes in (np.bool_(True), torch.tensor(True), 2):
        got = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu,
                                 interleaved=yes)
        assert torch.equal(got, q)
    for scale, shares in ((np.float32(0.125), np.int64(3)), (torch.tensor(0.125), np.int32(3)),
                          (np.float64(0.125), torch.tensor(3))):
        got = skv.kv_prefill_attn(c.kv, q, scale, cu_tokens=c.cu, num_shares=shares)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert_no_device_error()


# ------------------------------------------------------------------------- angles, positions

@pytest.mark.parametrize("packed", [True, False])
def test_angles_are_right_to_the_header_s_bound(packed):
    """Pairs (1, 0) become (cos, sin) of the angle, which is off by at most 2^-28 of a turn (the
    float) and 2^-32 (the fraction's cut); sincospif adds a unit, 2^-23 of the value. (1, 0) makes
    the products and the sum exact."""
    T, D = 4096, 64
    rng = np.random.default_rng(2)
    pos = np.concatenate([np.arange(1024), rng.integers(-2 ** 31, 2 ** 31, T - 1024)])
    c = Case((1,) * T if not packed else (T,), (0,) * (1 if packed else T), "fp32", D, 1, Hkv=1)
    c.q.copy_((torch.arange(D, device="cuda") < D // 2).float().expand_as(c.q))
    turns = skv.kv_rope_turns([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], device="cuda")
    stats = c.past_stats()
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu if packed else None,
                           positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert_no_device_error()
    frac = np.array([[(t % 2 ** 64) * int(p) % 2 ** 64 / 2.0 ** 64 for t in turns.tolist()]
                     for p in pos])
    angle = 2 * np.pi * np.where(frac > 0.5, frac - 1, frac)
    want = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    bound = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32) + 2.0 ** -23 * np.abs(want)
    err = np.abs(f64(q)[:, 0] - want)
    assert (err <= bound).all(), (err / bound).max()


# ------------------------------------------------------------------------ few rows, exactly

@pytest.mark.parametrize("new,past,D,G,PS,shares", [
    ((1,), (2047,), 128, 4, 16, 0),
    ((1, 1, 1, 1, 1, 1), (0, 1, 127, 128, 300, 1200), 128, 8, 16, 2),
    ((5, 5, 5), (63, 1500, 700), 64, 1, 16, 7),
    ((4, 4, 4), (63, 1500, 700), 128, 8, 64, 0),
    ((32, 31), (0, 900), 128, 1, 32, 40),
    ((8, 7), (0, 500), 64, 4, 64, 3),
    ((200,) + (1,) * 31, (100,) + (500,) * 31, 128, 4, 16, 0),
    ((301,) + (1,) * 31, (0,) + (300,) * 31, 64, 2, 32, 5),
    ((130, 0, 0, 2, 0), (0, 50, 0, 126, 0), 128, 1, 16, 0),
])
def test_few_rows_take_p_to_2_17(new, past, D, G, PS, shares):
    """A batch of at most 32 rows (tokens times group heads) to a sequence multiplies the values
    with P in two parts. A probability in [2^e, 2^(e+1)) is first off by at most 2^(e-8); what that
    leaves lies below that power, so its own half step is 2^(e-17) at most: 2^-17 together.
    Otherwise the bounds of the prompt attention: the row's own and the sum's logits, the
    exponential, sums over the keys, and the output's rounding."""
    c = Case(new, past, "bf16", D, G, PS=PS)
    assert sum(new) * G <= 32 * len(new) and shares != 1
    c.q.mul_(1.5)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=shares)
    assert_no_device_error()
    ref, ref_lse, mass, logit = prompt.prefill(f64(c.q), f64(c.k_pool), f64(c.v_pool),
                                               c.table.cpu().numpy(), c.lens, c.cu_h, PS, c.scale)
    rel = 2 * D * 2.0 ** -23 * logit + 2.0 ** -21 + max(c.lens) * 2.0 ** -23
    tol = (rel + 2.0 ** -17)[..., None] * mass * 1.01 + 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-30
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), (err / tol).max()
    assert (np.abs(f64(lse) - ref_lse) <= rel + 2.0 ** -23 * np.abs(ref_lse)).all()


def test_with_one_share_the_bits_do_not_depend_on_the_batch():
    """num_shares = 1 cuts no row's keys, and the batch's mean of rows chooses nothing there: a
    sequence alone, among single tokens and beside a prompt gives the same bits."""
    c = Case((1, 1, 500, 2), (900, 77, 30, 1300), "bf16", 128, 4)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, num_shares=1)
    for pick in ([0], [1], [3], [0, 1], [0, 3], [2]):
        rows = torch.cat([torch.arange(int(c.cu_h[b]), int(c.cu_h[b + 1])) for b in pick]).cuda()
        kv = skv.PagedKV(c.k_pool, c.v_pool, c.table[pick].contiguous(),
                         c.seq_lens[pick].contiguous())
        cu = torch.tensor(np.concatenate([[0], np.cumsum([c.new[b] for b in pick])]),
                          dtype=torch.int32, device="cuda")
        got, got_lse = skv.kv_prefill_attn(kv, c.q[rows].contiguous(), c.scale, cu_tokens=cu,
                                           num_shares=1)
        assert torch.equal(got, out[rows]) and torch.equal(got_lse, lse[rows])
        if all(c.new[b] == 1 for b in pick):
            got, got_lse = skv.kv_prefill_attn(kv, c.q[rows].contiguous(), c.scale, num_shares=1)
            assert torch.equal(got, out[rows]) and torch.equal(got_lse, lse[rows])
    assert_no_device_error()


@pytest.mark.parametrize("dtype,D,G,PS,rot,inter", [
    ("bf16", 128, 4, 16, 64, False), ("bf16", 128, 1, 32, 16, True), ("bf16", 64, 8, 64, 48, True),
    ("fp32", 128, 2, 16, 96, False), ("fp32", 64, 4, 32, 32, True),
])
@pytest.mark.parametrize("given", [True, False])
def test_one_token_with_part_of_the_head_rotated(dtype, D, G, PS, rot, inter, given):
    """The single-token form with fewer rotated columns than the head has, by the cache's
    positions and by positions given: the first past 2^31 in magnitude, negative and repeated."""
    past = (0, 15, 16, 31, 100, 63)
    c = Case((1,) * len(past), past, dtype, D, G, PS=PS)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -7, 12345, 12345, 0])
    stats = c.past_stats()
    before = (c.k_pool.clone(), c.v_pool.clone(), None)
    c.q_in = c.q.clone()
    turns = skv.kv_rope_turns(freqs(rot), device="cuda")
    where = torch.tensor(pos, dtype=torch.int32, device="cuda") if given else None
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, interleaved=inter, positions=where)
    assert_no_device_error()
    check_append(c, q, stats, before, rot, inter, pos_of_row=pos if given else None)
    mapped = pages_of(c, c.lens)
    rebuilt = skv.kv_build_page_stats(c.kv)
    np.testing.assert_array_equal(f64(stats)[mapped], f64(rebuilt)[mapped])


@pytest.mark.parametrize("new", [(20, 1, 300), (1, 1, 1)])
def test_append_statistics_past_32_bit_offsets(new):
    """Statistics of more than 2^31 elements: those of the last pages are joined with what was
    there and equal the same call's on a small cache; the first pages stay as they were."""
    packed = new[0] > 1
    c = Case(new, (5, 16, 40), "bf16", 128, 4, Hkv=2, PS=16, extra=0)
    need = c.k_pool.shape[0]
    NP = 2 ** 31 // (2 * 2 * 128) + need + 8
    if torch.cuda.mem_get_info()[0] < 90 * 2 ** 30:
        pytest.skip("needs 74 GB of device memory")
    turns = skv.kv_rope_turns(freqs(128), device="cuda")
    stats = c.past_stats()
    k = torch.empty((NP, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    far = torch.empty((NP, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    for big, small in ((k, c.k_pool), (v, c.v_pool), (far, stats)):
        big[-need:] = small
        big[:64] = 3.0
    table = torch.where(c.table >= 0, c.table + (NP - need), c.table).to(torch.int32)
    cu = c.cu if packed else None
    q_far = skv.kv_append_rope(skv.PagedKV(k, v, table, c.seq_lens), c.q, c.k, c.v, far, turns,
                               cu_tokens=cu)
    q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=cu)
    assert_no_device_error()
    assert torch.equal(q_far, q)
    used = pages_of(c, c.lens)
    for big, small in ((k, c.k_pool), (v, c.v_pool), (far, stats)):
        assert torch.equal(big[-need:][used], small[used])
        assert (big[:64] == 3.0).all()
    np.testing.assert_array_equal(f64(stats[used]), f64(skv.kv_build_page_stats(c.kv)[used]))


# ------------------------------------------------------------------- keys that are not numbers

@pytest.mark.parametrize("dtype,D,PS,many", [("bf16", 128, 16, False), ("bf16", 64, 64, False),
                                             ("fp32", 128, 32, False), ("fp32", 64, 16, False),
                                             ("bf16", 128, 64, True), ("bf16", 128, 16, True)])
def test_statistics_of_keys_with_nan_equal_the_full_build_s(dtype, D, PS, many):
    """A NaN in a page's first key stays, one in a later key does not count, and infinities are
    extremes: in pages that begin with the call, resume a page or are filled one by one."""
    new = (2500, 1700, 70) if many else (100, 70, 1)
    c = Case(new, (0, 5, PS), dtype, D, 2, Hkv=2, PS=PS)
    k = c.k                                                # a view into the fused rows
    gen = torch.Generator(device="cuda").manual_seed(8)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(k.dtype)
    pick = torch.randint(0, 12, k.shape, generator=gen, device="cuda")
    for i in range(3):
        k[pick == i] = bad[i]
    k[:, :, 3] = float("nan")                              # a column without any number
    k[:, 0, 5] = float("inf")
    c.k_pool[c.table[1, 0].long(), :, 0, 7] = float("nan")  # held by a page before the call
    stats = c.past_stats()
    skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, cu_tokens=c.cu)
    assert_no_device_error()
    table = c.table.flatten().long()
    used = table[table >= 0]
    rebuilt = skv.kv_build_page_stats(c.kv)
    np.testing.assert_array_equal(f64(stats[used]), f64(rebuilt[used]))
    assert torch.isnan(stats[used]).any()


# ---------------------------------------------------------------------- streams by argument

def busy(stream):
    """Work of some milliseconds on a stream, so that what follows there runs after the host's."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(10_000_000)


def test_attention_on_streams_given_by_argument():
    """Buffers that the call makes for itself belong to its stream: the current stream's later
    allocations and writes do not touch them, nor do two calls on two streams share one."""
    c = Case((200, 31, 1), (100, 900, 4000), "bf16", 128, 4)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu)
    nbytes = skv.kv_prefill_attn_workspace_size(c.kv, c.Hq, c.T)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s in streams:
            busy(s)
        for s in streams:
            got.append(skv.kv_prefill_attn(c.kv, c.q, c.scale, cu_tokens=c.cu, stream=s))
        for n in (nbytes, ref.numel() * 2, ref_lse.numel() * 4):
            for _ in range(3):                # what the allocator would hand out again
                torch.empty((n,), dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert_no_device_error()
        for out, lse in got:
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_append_on_a_stream_given_by_argument():
    """The rotated queries' buffer is the stream's: not one that the current stream still uses."""
    c = Case((40, 3), (9, 30), "bf16", 128, 4, PS=16)
    turns = skv.kv_rope_turns([0.5] * 64, device="cuda")
    stats = c.past_stats()
    ref = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu)
    k1, s1 = c.k_pool.clone(), stats.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        old = torch.empty_like(ref)           # freed with a write of this stream still to come
        torch.cuda._sleep(10_000_000)
        old.fill_(7.0)
        del old
        q = skv.kv_append_rope(c.kv, c.q, c.k, c.v, stats, turns, cu_tokens=c.cu, stream=s)
        torch.cuda.synchronize()
        assert_no_device_error()
        assert torch.equal(q, ref) and torch.equal(c.k_pool, k1) and torch.equal(stats, s1)
        del q


# ------------------------------------------------------------------ waits that run out

def long_items(D, tokens, Hkv=2):
    """One row per sequence over a table that names the same few pages again and again: the KV
    heads are items of tokens / 128 key tiles each, one after the other with num_shares = 1."""
    c = Case((1,), (200,), "bf16", D, 4, Hkv=Hkv, PS=64)
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
def test_waits_of_few_rows_that_run_out_are_flagged_too(wait_limit, D):
    """The same where P has two parts: two shares of eight KV heads, several items to a block."""
    c = long_items(D, 1 << 22, Hkv=8)
    ref, ref_lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=2)
    assert_no_device_error()
    for limit, want in ((0, (-6, 16)), (50_000, (0, 0)), (0, (-6, 16))):
        wait_limit(limit)
        out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=2)
        wait_limit(2_000_000_000)
        assert skv.kv_check_device_errors() == want
        if want == (0, 0):
            assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out, lse = skv.kv_prefill_attn(c.kv, c.q, c.scale, num_shares=2)
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
