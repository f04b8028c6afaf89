"""Oracle of the page operators, token by token and page by page (test infrastructure only)."""

from __future__ import annotations

import numpy as np


def compact(k_pool, v_pool, table, seq_lens, counts, kept, page_size):
    """Moves the tokens ``kept[b]`` of sequence b's last ``counts[b]`` ones together, on copies of
    the pools: (k_pool, v_pool, new lengths, touched), ``touched`` the (sequence, page) pairs whose
    statistics are taken anew."""
    k, v = np.array(k_pool), np.array(v_pool)
    lens, touched = [], []
    for b, keep in enumerate(kept):
        start = int(seq_lens[b]) - int(counts[b])
        rows = [(k_pool[table[b][t // page_size], :, t % page_size],
                 v_pool[table[b][t // page_size], :, t % page_size])
                for t in (start + j for j in keep)]
        for i, (kr, vr) in enumerate(rows):
            P, slot = table[b][(start + i) // page_size], (start + i) % page_size
            k[P, :, slot], v[P, :, slot] = kr, vr
        lens.append(start + len(keep))
        if counts[b]:
            touched += [(b, p) for p in range(start // page_size, -(-lens[b] // page_size))]
    return k, v, lens, touched


def update_pages(table, lens, refs, rows, parents, keep, want, page_size, window=0, sinks=0):
    """The next page table by the rules of the call, one entry at a time: (table, refs, copies,
    free_left). ``table`` [old rows][stride], ``parents`` a list or None."""
    stride = table.shape[1]
    refs = [int(r) for r in refs]
    out = np.full((rows, stride), -1, dtype=np.int64)
    parents = list(range(rows)) if parents is None else parents
    for b in range(rows):
        if parents[b] < 0:
            continue
        assert 0 <= keep[b] <= lens[parents[b]]
        for p in range(-(-keep[b] // page_size)):
            gone = window > 0 and p * page_size >= sinks and \
                (p + 1) * page_size <= keep[b] - window + 1
            if not gone:
                out[b, p] = table[parents[b], p]
    for old, sign in ((out, 1), (table, -1)):
        for P in old.ravel():
            if P >= 0:
                refs[P] += sign
    held = refs[:]
    # rows that write to a partial page, and the holders of it that do not
    writes = {}
    for b in range(rows):
        if want[b] > keep[b] and keep[b] % page_size and out[b, keep[b] // page_size] >= 0:
            writes.setdefault(int(out[b, keep[b] // page_size]), []).append(b)
    copying = {}
    for P, who in writes.items():
        others = refs[P] - len(who)
        for b in who if others > 0 else who[:-1]:
            copying[b] = P
            refs[P] -= 1
    free = [P for P, r in enumerate(refs) if r == 0]
    needs = [-(-want[b] // page_size) - -(-keep[b] // page_size) + (b in copying)
             for b in range(rows)]
    copies = np.full((rows, 2), -1, dtype=np.int64)
    if sum(needs) > len(free):
        return out, held, copies, len(free) - sum(needs)
    left = len(free) - sum(needs)
    for b in range(rows):
        first = -(-keep[b] // page_size)
        if b in copying:
            fresh = free.pop(0)
            copies[b] = copying[b], fresh
            out[b, first - 1] = fresh
            refs[fresh] = 1
        for p in range(first, -(-want[b] // page_size)):
            fresh = free.pop(0)
            out[b, p] = fresh
            refs[fresh] = 1
    return out, refs, copies, left
