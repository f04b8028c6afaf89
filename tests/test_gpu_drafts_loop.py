"""The calls for drafts, windows and pages together, as a server runs them: sequences come, fork,
verify trees of drafts, keep some of them and go, over the caches of two layers that share a page
table. What the caches hold is followed on the host token by token."""

import random

import numpy as np
import pytest
import torch

import sparse_kv_cache_build_gb300 as skv
from oracle import prompt

from gpu_helpers import assert_no_device_error, f64, need_gpu
from test_gpu_prompt import freqs, half_step

pytestmark = pytest.mark.gpu

HKV, G, D, PS, NP, STRIDE = 2, 4, 64, 16, 400, 40
LAYERS = 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    torch.cuda.set_device(0)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """The device state, and beside it what every sequence holds: per token its key and value rows
    of each layer, as bits."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (NP, HKV, PS, D)
        bad = dict(fill_value=float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pools = [(torch.full(shape, **bad), torch.full(shape, **bad)) for _ in range(LAYERS)]
        self.stats = [torch.full((NP, HKV, 2, D), **bad) for _ in range(LAYERS)]
        self.refs = torch.zeros(NP, dtype=torch.int32, device="cuda")
        self.table, self.lens = ints([[-1] * STRIDE]), [0]
        self.turns = skv.kv_rope_turns(freqs(D), device="cuda")
        self.held = [[]]

    def caches(self):
        lens = ints(self.lens)
        return [skv.PagedKV(k, v, self.table, lens) for k, v in self.pools]

    def update(self, want, keep, parents=None, **kw):
        self.table, copies, left = skv.kv_update_pages(
            self.caches()[0], self.refs, ints(want), keep_lens=ints(keep),
            parents=None if parents is None else ints(parents), **kw)
        self.lens = list(want)
        for kv, stats in zip(self.caches(), self.stats):
            skv.kv_copy_pages(kv, copies, stats)
        parents = range(len(want)) if parents is None else parents
        self.held = [self.held[p][:k] if p >= 0 else [] for p, k in zip(parents, keep)]
        return int(left)

    def append(self, rows, positions):
        """The last rows[b] tokens of each sequence, at the given positions: queries per layer."""
        T = sum(rows)
        cu = ints(np.concatenate([[0], np.cumsum(rows)]).tolist())
        queries, keys = [], []
        for kv, stats in zip(self.caches(), self.stats):
            x = torch.randn((T, HKV * G + 2 * HKV, D), generator=self.gen, device="cuda")
            q, k, v = x.to(torch.bfloat16).split((HKV * G, HKV, HKV), dim=1)
            queries.append(skv.kv_append_rope(kv, q, k, v, stats, self.turns, cu_tokens=cu,
                                              positions=ints(positions)))
            turned, _ = prompt.rope(f64(k), positions, freqs(D))
            keys.append((turned, f64(v)))
        at = 0
        for b, n in enumerate(rows):
            for i in range(n):
                self.held[b].append((positions[at + i],
                                     [(k[at + i], v[at + i]) for k, v in keys]))
            at += n
        return queries, cu

    def check(self, gone=lambda b, t: False):
        """Every sequence's tokens are where the table says, and the statistics are theirs."""
        table = self.table.cpu().numpy()
        for layer, (kv, (kp, vp)) in enumerate(zip(self.caches(), self.pools)):
            kp, vp = f64(kp), f64(vp)
            for b, tokens in enumerate(self.held):
                assert len(tokens) == self.lens[b]
                for t, (_, rows) in enumerate(tokens):
                    if gone(b, t):
                        continue
                    P = table[b, t // PS]
                    k, v = rows[layer]
                    # rounded to bf16 after a rotation in 32 bits (test_gpu_prompt.py)
                    tol = half_step("bf16") * np.abs(k) + 2.0 ** -21 * 2 * np.abs(k).max() + 1e-6
                    assert (np.abs(kp[P, :, t % PS] - k) <= 1.01 * tol).all()
                    assert np.array_equal(vp[P, :, t % PS], v)
        used = table[table >= 0]
        assert np.array_equal(np.bincount(used, minlength=NP), self.refs.cpu().numpy())

    def check_stats(self):
        used = sorted({int(self.table[b, p]) for b, n in enumerate(self.lens)
                       for p in range(-(-n // PS))})
        for kv, stats in zip(self.caches(), self.stats):
            assert torch.equal(stats[used], skv.kv_build_page_stats(kv)[used])

    def attention(self, layer, b, q, hidden):
        """64-bit attention of rows q over sequence b as the pool holds it."""
        K, V = (prompt.cached_rows(f64(x), self.table.cpu().numpy(), b, self.lens[b], PS)
                for x in self.pools[layer])
        out = np.empty(q.shape)
        mass = np.empty(q.shape)
        for h in range(HKV * G):
            z = q[:, h] @ K[:, h // G].T * D ** -0.5
            z[hidden] = -np.inf
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[:, h], mass[:, h] = p @ V[:, h // G], p @ np.abs(V[:, h // G])
        # P to bf16 (2^-8 at most), the output's rounding, and 2^-13 for logits of up to 64 columns
        return out, 1.01 * ((half_step("bf16") + 2.0 ** -13) * mass + half_step("bf16") *
                            np.abs(out))


def tree_of(rng, n):
    up = [-1 if i == 0 or rng.random() < 0.2 else rng.randrange(max(0, i - 4), i)
          for i in range(n)]
    depth = []
    for p in up:
        depth.append(0 if p < 0 else depth[p] + 1)
    return up, depth


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_drafts_forks_and_windows(seed):
    rng = random.Random(seed)
    s = Server(seed)
    # prompts
    first = [rng.randrange(1, 130) for _ in range(3)]
    assert s.update(first, [0] * 3, parents=[-1] * 3) > 0
    queries, cu = s.append(first, [t for n in first for t in range(n)])
    s.check()
    for step in range(4):
        # trees of drafts are appended and verified
        past = list(s.lens)
        trees = [tree_of(rng, rng.choice((1, 5, 12, 19))) for _ in past]
        rows = [len(up) for up, _ in trees]
        assert s.update([p + n for p, n in zip(past, rows)], past) > 0
        parents = ints([p for up, _ in trees for p in up])
        queries, cu = s.append(rows, [p + d for p, (_, depth) in zip(past, trees) for d in depth])
        for layer, kv in enumerate(s.caches()):
            out, lse = skv.kv_tree_attn(kv, queries[layer], D ** -0.5, parents, cu_tokens=cu)
            at = 0
            for b, (up, _) in enumerate(trees):
                ref, tol = s.attention(layer, b, f64(queries[layer][at:at + rows[b]]),
                                       prompt.tree_hidden(up, s.lens[b]))
                assert (np.abs(f64(out[at:at + rows[b]]) - ref) <= tol).all()
                at += rows[b]
        # the way to one node is accepted
        kept = []
        for up, _ in trees:
            way, node = [], rng.randrange(-1, len(up))
            while node >= 0:
                way.insert(0, node)
                node = up[node]
            kept.append(way)
        most = max(1, max(map(len, kept)))
        keep, cnt = ints([k + [0] * (most - len(k)) for k in kept]), ints([len(k) for k in kept])
        for kv, stats in zip(s.caches(), s.stats):
            lens = skv.kv_compact(kv, keep, cnt, stats, cu_tokens=cu)
        s.held = [h[:p] + [h[p + j] for j in k] for h, p, k in zip(s.held, past, kept)]
        s.lens = lens.tolist()
        for b, tokens in enumerate(s.held):               # an accepted way is a line of positions
            assert [pos for pos, _ in tokens] == list(range(len(tokens)))
        # pages of dropped drafts go back; sequences fork, come and go
        order = [rng.randrange(-1, len(s.lens)) for _ in range(rng.choice((2, 3, 5)))]
        lens = [s.lens[p] if p >= 0 else 0 for p in order]
        assert s.update(lens, lens, parents=order) > 0
        s.check()
        fresh = [1 + (0 if p >= 0 else rng.randrange(40)) for p in order]
        assert s.update([n + f for n, f in zip(lens, fresh)], lens) > 0
        s.append(fresh, [n + i for n, f in zip(lens, fresh) for i in range(f)])
        s.check()
        s.check_stats()
    # streams: a window of 40 tokens and three sinks, a token at a time
    window, sinks = 40, 3
    for step in range(20):
        past = list(s.lens)
        assert s.update([p + 1 for p in past], past, window=window, sinks=sinks) > 0
        queries, cu = s.append([1] * len(past), past)
        # what pages outside still hold is not the rows' concern
        s.check(gone=lambda b, t: int(s.table[b, t // PS]) < 0)
        if step % 5:
            continue
        for layer, kv in enumerate(s.caches()):
            out, lse = skv.kv_window_attn(kv, queries[layer], D ** -0.5, window, sinks)
            for b, n in enumerate(s.lens):
                pos = np.array([u for u in range(n) if u > n - 1 - window or u < sinks])
                K, V = (np.stack([f64(x[int(s.table[b, u // PS]), :, u % PS]) for u in pos])
                        for x in s.pools[layer])
                q = f64(queries[layer][b])
                for h in range(HKV * G):
                    z = K[:, h // G] @ q[h] * D ** -0.5
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    ref, mass = p @ V[:, h // G], p @ np.abs(V[:, h // G])
                    tol = 1.01 * ((half_step("bf16") + 2.0 ** -13) * mass +
                                  half_step("bf16") * np.abs(ref))
                    assert (np.abs(f64(out[b, h]) - ref) <= tol).all()
    s.update([0], [0], parents=[-1])
    assert int(s.refs.sum()) == 0
    assert_no_device_error()


def test_dropped_tokens_leave_the_statistics():
    """A page whose last tokens are dropped: its statistics follow by a compaction that keeps none
    of them, and the next append builds on them."""
    s = Server(5)
    assert s.update([45, 30], [0, 0], parents=[-1, -1]) > 0
    s.append([45, 30], list(range(45)) + list(range(30)))
    drop = ints([0, 9, 9 + 14])
    for kv, stats in zip(s.caches(), s.stats):
        lens = skv.kv_compact(kv, ints([[0], [0]]), ints([0, 0]), stats, cu_tokens=drop)
    assert lens.tolist() == [36, 16]
    s.held, s.lens = [h[:n] for h, n in zip(s.held, (36, 16))], [36, 16]
    s.check_stats()
    assert s.update([40, 17], [36, 16]) > 0
    s.append([4, 1], [36, 37, 38, 39, 16])
    s.check()
    s.check_stats()
    assert_no_device_error()
