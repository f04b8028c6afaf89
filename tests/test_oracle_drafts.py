"""Pins of the oracles for drafts, windows and pages: masks against other statements of them, page
tables against what they have to keep."""

import random

import numpy as np

from oracle import pages, prompt


def test_a_window_mask_counts_what_is_left():
    for n, length, window, sinks in ((1, 1, 1, 0), (5, 9, 3, 2), (9, 9, 4, 0), (4, 30, 7, 40)):
        hidden = prompt.window_hidden(n, length, window, sinks)
        for i in range(n):
            pos = length - n + i
            seen = np.flatnonzero(~hidden[i])
            first = set(range(min(sinks, pos + 1)))
            last = set(range(max(0, pos - window + 1), pos + 1))
            assert set(seen) == first | last


def test_a_tree_mask_is_reachability():
    rng = np.random.default_rng(1)
    for n in (1, 2, 17, 40):
        up = [-1 if i == 0 or rng.random() < 0.2 else int(rng.integers(0, i)) for i in range(n)]
        step = np.eye(n, dtype=int)
        for i, p in enumerate(up):
            if p >= 0:
                step[i, p] = 1
        reach = np.linalg.matrix_power(step, n) > 0
        hidden = prompt.tree_hidden(up, n + 5)
        assert not hidden[:, :5].any()
        np.testing.assert_array_equal(~hidden[:, 5:], reach)


def test_masked_rows_are_rows_over_what_they_see():
    rng = np.random.default_rng(2)
    PS, D = 16, 64
    table = np.arange(4).reshape(1, 4)
    K, V = rng.normal(size=(4, 1, PS, D)), rng.normal(size=(4, 1, PS, D))
    q = rng.normal(size=(6, 2, D))
    lens, cu = np.array([50]), np.array([0, 6])
    out, lse, mass, logit = prompt.prefill(
        q, K, V, table, lens, cu, PS, 0.125,
        hidden_of=lambda b, n, length: prompt.window_hidden(n, length, 9, 3))
    k, v = K.transpose(0, 2, 1, 3).reshape(-1, D), V.transpose(0, 2, 1, 3).reshape(-1, D)
    for i in range(6):
        pos = 44 + i
        at = [u for u in range(pos + 1) if u > pos - 9 or u < 3]
        for h in range(2):
            z = 0.125 * k[at] @ q[i, h]
            p = np.exp(z)
            np.testing.assert_allclose(out[i, h], p @ v[at] / p.sum(), atol=1e-12)
            np.testing.assert_allclose(lse[i, h], np.log(p.sum()), atol=1e-12)


def test_compaction_of_rising_lists():
    """Against a plain list of tokens per sequence."""
    rng = random.Random(3)
    PS, lens, counts = 4, [13, 7, 20], [6, 0, 20]
    table = np.array([[0, 5, 1, 9, -1], [2, 3, -1, -1, -1], [4, 6, 7, 8, 10]])
    pool = np.arange(11 * PS, dtype=float).reshape(11, 1, PS, 1)
    kept = [sorted(rng.sample(range(n), n // 2)) for n in counts]
    k, v, new, touched = pages.compact(pool, -pool, table, lens, counts, kept, PS)

    def tokens(x, b, n):
        return [x[table[b, t // PS], 0, t % PS, 0] for t in range(n)]

    for b in range(3):
        before = tokens(pool, b, lens[b])
        start = lens[b] - counts[b]
        want = before[:start] + [before[start + j] for j in kept[b]]
        assert tokens(k, b, new[b]) == want and tokens(v, b, new[b]) == [-x for x in want]
        assert len(want) == new[b]
    assert {b for b, _ in touched} == {0, 2}


def test_page_tables_keep_their_counts_and_their_tokens():
    """Over random steps: an entry is held as often as it is counted, a page that a row may write
    to is its own, and a kept token stays where a copy says."""
    rng = random.Random(0)
    for trial in range(60):
        NP, stride, PS = 60, 8, 4
        table, lens, refs = np.full((1, stride), -1), [0], [0] * NP
        content = {}                                  # (page, slot) -> token id
        held = [[]]
        for step in range(15):
            rows = rng.choice((1, 2, 5))
            parents = None if rng.random() < 0.3 else \
                [rng.randrange(-1, len(lens)) for _ in range(rows)]
            src = list(range(len(lens))) if parents is None else parents
            old = [lens[q] if q >= 0 else 0 for q in src]
            keep = [max(0, x - rng.choice((0, 0, 1, 5))) for x in old]
            want = [min(stride * PS, k + rng.choice((0, 1, 3, 9))) for k in keep]
            table, refs, copies, left = pages.update_pages(table, lens, refs, len(want), parents,
                                                           keep, want, PS)
            used = table[table >= 0]
            assert np.array_equal(np.bincount(used, minlength=NP), refs)
            assert left < 0 or left == refs.count(0)
            held = [held[q][:k] if q >= 0 else [] for q, k in zip(src, keep)]
            if left < 0:
                lens = keep
                continue
            for a, b in copies:
                for s in range(PS):
                    if a >= 0 and (a, s) in content:
                        content[b, s] = content[a, s]
            for b in range(len(want)):
                for t in range(keep[b], want[b]):
                    assert refs[table[b, t // PS]] == 1
                    content[table[b, t // PS], t % PS] = (trial, step, b, t)
                    held[b].append((trial, step, b, t))
            for b, tokens in enumerate(held):
                assert [content[table[b, t // PS], t % PS] for t in range(len(tokens))] == tokens
            lens = want
